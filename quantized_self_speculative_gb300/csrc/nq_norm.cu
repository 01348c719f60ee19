// nq_norm.cu -- root-mean-square norm between two linears: the residual's
// addition before it, bf16 activations or int8 codes with row scales after it.
//
//   s = x + a (rounded once to x's type, stored);  y = s rsqrt(mean(s^2) + eps) w
//   codes: z = max|y| / 127, clamp(rint(y / z), -127, 127), as nq_quantize_act_int8
//
// One CTA takes a row and holds it in registers: x, a and w are read once, two
// block reductions (the second for codes only), one write.  The codes come from
// the fp32 y, which is never rounded to bf16 on the way.  Sums of squares are
// taken in fp32: four neighbours in a chain, four such groups (a quarter of the row
// apart) in order, then a tree.
// Many rows: a thread takes four groups, so that loads in flight cover the latency;
// few rows: one group and four times the threads, which add up in the same order, so
// that a row gives the same bits either way.  Bound by HBM, and by latency for few rows.
// Measured (GB300): 16381 rows of 3584, bf16 residual + fp32, bf16 out: 92 us, 6.4 TB/s (94% of the
// copy rate; with two groups per thread 108, with one 140); codes out 106 us, 5.0 TB/s (73%), from fp32
// rows 113 us, 6.8 TB/s.  Rows of few values leave most of a CTA's one warp idle: 100000 of 128 take
// 55 us (bf16 out, 0.9 TB/s) and 70 (codes), as many of 64 the same.
#include "nq_internal.cuh"

namespace nq {
namespace {

struct NormArgs {
    const void *x, *a, *w;
    long long xs, as, ss;     // elements between rows
    void *sum;
    uint16_t *y;
    int8_t *xq;
    float *sx;
    int K, threads;
    bool a_bf16, w_bf16;
    float eps;
    unsigned int *status;
};

__device__ __forceinline__ float max_nan(float a, float b)      // NaN where either is
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void widen(float (&v)[4], uint2 u)
{
    v[0] = __uint_as_float(u.x << 16);
    v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16);
    v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(float (&v)[4], const void *p, long long at, bool bf16)
{
    if (bf16) {
        widen(v, *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at));
    } else {
        const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    }
}
// Over the first `threads` threads, whole warps; every thread of the CTA gets the result.  `red` holds a float per
// warp and is not in use by others.
template <bool MAX>
__device__ __forceinline__ float over_block(float v, int threads, float *red)
{
    auto join = [](float a, float b) { return MAX ? max_nan(a, b) : a + b; };
    if (threadIdx.x < threads) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < threads >> 5 ? red[lane] : 0.0f;                  // 0: below every |y|, nothing in a sum
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Groups of four neighbours: thread t of A.threads takes groups t, t + threads, + 2, + 3 threads; NV = 1: four threads
// (t, t + threads, ..) take one each.
template <int NV, bool XB>
__global__ void __launch_bounds__(1024)
norm_kernel(const __grid_constant__ NormArgs A)
{
    __shared__ float red[2][32], part[NV == 1 ? 1024 : 1];
    const long long row = blockIdx.x;
    const int groups = A.K >> 2, step = A.threads;              // (NV = 1: threadIdx.x runs over all four quarters)
    float v[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = threadIdx.x + i * step;
        v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.0f;
        if (g < groups) load4(v[i], A.x, row * A.xs + 4 * g, XB);
    }
    if (A.a) {
        float a[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int g = threadIdx.x + i * step;
            a[i][0] = a[i][1] = a[i][2] = a[i][3] = 0.0f;
            if (g < groups) load4(a[i], A.a, row * A.as + 4 * g, A.a_bf16);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int g = threadIdx.x + i * step;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] += a[i][e];
            if constexpr (XB) {
                const uint2 u = make_uint2(pair_bf16(v[i][0], v[i][1]), pair_bf16(v[i][2], v[i][3]));
                widen(v[i], u);
                if (g < groups) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(A.sum) + row * A.ss + 4 * g) = u;
            } else if (g < groups) {
                *reinterpret_cast<float4 *>(static_cast<float *>(A.sum) + row * A.ss + 4 * g) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
            }
        }
    }
    float w[NV][4];           // asked for before the reduction's wait
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = threadIdx.x + i * step;
        w[i][0] = w[i][1] = w[i][2] = w[i][3] = 1.0f;
        if (A.w && g < groups) load4(w[i], A.w, 4 * g, A.w_bf16);
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fmaf(v[i][e], v[i][e], s);
        ss = i == 0 ? s : ss + s;
    }
    if constexpr (NV == 1) {
        part[threadIdx.x] = ss;
        __syncthreads();
        if (threadIdx.x < step)
            for (int i = 1; i < 4; ++i) ss += part[threadIdx.x + i * step];
    }
    ss = over_block<false>(ss, step, red[0]);
    const bool finite = ss <= 3.4028235e38f;
    if (!finite && threadIdx.x == 0) set_status(A.status, NQ_DEV_NONFINITE);
    const float f = rsqrtf(__fdiv_rn(ss, static_cast<float>(A.K)) + A.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = v[i][e] * f * w[i][e];
    if (A.y) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int g = threadIdx.x + i * step;
            if (g < groups)
                *reinterpret_cast<uint2 *>(A.y + row * A.K + 4 * g) = make_uint2(pair_bf16(v[i][0], v[i][1]), pair_bf16(v[i][2], v[i][3]));
        }
    }
    if (!A.xq) return;
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max_nan(top, fabsf(v[i][e]));
    top = over_block<true>(top, blockDim.x, red[1]);
    float z = __fdiv_rn(top, 127.0f);
    if (!finite || !(top <= 3.4028235e38f)) {
        if (finite && threadIdx.x == 0) set_status(A.status, NQ_DEV_NONFINITE);   // the weight's doing
        z = 0.0f;
    }
    if (threadIdx.x == 0) A.sx[row] = z;
    // y / z by Markstein's correction: a product with the rounded 1 / z, and its error taken off in fused operations.  That is
    // the quotient but for 2^-46 of it, rounded once, so that it could differ from the division's only within 2^-46 of the
    // middle between two fp32 numbers; no code does, at any border k + 1/2 and any mantissa of z (all were tried).  The
    // error's unit, 2^-48 z beside a border, is a fp32 number from z = 1e-30 on.  (Division: 100 us instead of 70 for 100000 rows of 128.)
    const float rz = __frcp_rn(z);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = threadIdx.x + i * step;
        uint32_t c = 0;
        if (z > 0.0f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float q0 = v[i][e] * rz, x = z < 1e-30f ? __fdiv_rn(v[i][e], z) : fmaf(fmaf(-q0, z, v[i][e]), rz, q0);
                const int q = static_cast<int>(fminf(fmaxf(rintf(x), -127.0f), 127.0f));
                c |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * e);
            }
        }
        if (g < groups) *reinterpret_cast<uint32_t *>(A.xq + row * A.K + 4 * g) = c;
    }
}

template <int NV>
void launch(const NormArgs &A, bool xb, int M, int threads, cudaStream_t s)
{
    if (xb) norm_kernel<NV, true><<<M, threads, 0, s>>>(A);
    else norm_kernel<NV, false><<<M, threads, 0, s>>>(A);
}

}  // namespace
}  // namespace nq

extern "C" nq_status nq_rms_norm(const void *x, int x_dtype, int64_t x_stride, const void *add, int add_dtype, int64_t add_stride,
                                 const void *weight, int w_dtype, float eps, int M, int K, void *sum, int64_t sum_stride,
                                 uint16_t *y, int8_t *xq, float *sx, cudaStream_t stream)
{
    auto known = [](int t) { return t == NQ_F32 || t == NQ_BF16; };
    if (!x || M < 1 || K < 1 || !known(x_dtype) || !(eps > 0.0f && eps <= 3.4028235e38f)) return NQ_ERR_ARG;
    if ((add && !known(add_dtype)) || (weight && !known(w_dtype)) || (add != nullptr) != (sum != nullptr)) return NQ_ERR_ARG;
    if ((!y && !xq) || (xq != nullptr) != (sx != nullptr)) return NQ_ERR_ARG;
    if (K % 8 != 0 || K > 16384) return NQ_ERR_SHAPE;
    auto rows = [&](int64_t s) { return s >= K && s % 8 == 0; };
    if (!rows(x_stride) || (add && (!rows(add_stride) || !rows(sum_stride)))) return NQ_ERR_SHAPE;
    if (!nq::aligned16(x) || !nq::aligned16(add) || !nq::aligned16(weight) || !nq::aligned16(sum) || !nq::aligned16(y) ||
        !nq::aligned16(xq) || (reinterpret_cast<uintptr_t>(sx) & 3u))
        return NQ_ERR_ALIGN;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    const int groups = K / 4, threads = ((groups + 3) / 4 + 31) / 32 * 32;
    const nq::NormArgs A{x, add, weight, x_stride, add_stride, sum_stride, sum, y, xq, sx, K, threads, add_dtype == NQ_BF16, w_dtype == NQ_BF16, eps, status};
    const bool xb = x_dtype == NQ_BF16;
    // one group per thread while the rows do not fill the GPU and 1024 threads hold one: 8.3 us against 10.4 for one row of
    // 4096 to codes and a product after it (144 rows: 10.3 either way)
    if (M <= 2 * nq::sm_count() && threads <= 256) nq::launch<1>(A, xb, M, 4 * threads, stream);
    else nq::launch<4>(A, xb, M, threads, stream);
    return nq::cuda_status(cudaGetLastError());
}
