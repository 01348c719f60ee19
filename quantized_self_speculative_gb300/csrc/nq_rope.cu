// nq_rope.cu -- rotary positions, and storing / reading rows of the paged KV
// cache (rotated, then quantised or rounded, in one pass over a fused linear's
// output).
//
// A pair turns by a = pos * w.  The rate w / (2 pi) is a 64-bit fraction of a
// turn, so frac(pos * rate) is one integer product: no precision is lost at
// far positions, and no table of angles is read.  sin and cos of that fraction
// are taken once per token and lane and used for every head that the warp handles.
//
// One warp takes one token and a run of heads, kBatch rows at a time: all their
// loads are issued before the first row is turned.  Lane l holds elements
// E l .. E l + E - 1 (E = D / 32) of a row, so an interleaved pair lies in one
// lane and a half pair is one shuffle away.
//
// Measured (GB300, 2070 MHz).  Rotation, 16384 tokens x 32 heads x 128, bf16 to
// bf16: 43.5 us, 6.2 TB/s, HBM bound (91% of the copy rate; fp32 in and out 83 us,
// 95%).  Append, 8191 tokens, 32 + 32 + 32 heads x 128, fp32 to nested groups of 64:
// 109 us, 5.0 TB/s, bound by instruction issue (some 110 warp instructions per row:
// maximum over the group, two correctly rounded quotients, the codes); to bf16
// pages 94 us (95%).  Read of the same rows: 44 us, 4.6 TB/s, bound by latency:
// 64-byte pieces of four heads at a time; from bf16 pages 47 us (84%).  A small call
// (144 tokens, 48 heads) takes 4.9 us, its read 2.3 us, one launch each.
#include <cmath>

#include "nq_page.cuh"

namespace nq {
namespace {

constexpr int kWarps = 4;               // short CTAs end together: append of 8191 tokens 3% faster than with 8

struct Rope {
    int rot, layout;
    float mscale, mscale_lo;
    const unsigned long long *rates;
};

template <int E> struct Vec { float v[E]; };

__device__ __forceinline__ void bf_pair(uint32_t w, float &a, float &b)
{
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
}
// A lane's E values as loaded; kBatch of them are in flight at once (16 registers).
template <int E, typename T> struct Raw;
template <int E>
struct Raw<E, float> {
    static constexpr int kBatch = 16 / E;
    float v[E];
    __device__ __forceinline__ void load(const float *p)
    {
        if constexpr (E == 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p);
            v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
            const float2 f = *reinterpret_cast<const float2 *>(p);
            v[0] = f.x; v[1] = f.y;
        }
    }
    __device__ __forceinline__ Vec<E> values() const
    {
        Vec<E> r;
#pragma unroll
        for (int e = 0; e < E; ++e) r.v[e] = v[e];
        return r;
    }
};
template <int E>
struct Raw<E, __nv_bfloat16> {
    static constexpr int kBatch = 8;
    uint32_t v[E / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        if constexpr (E == 4) {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            v[0] = w.x; v[1] = w.y;
        } else {
            v[0] = *reinterpret_cast<const uint32_t *>(p);
        }
    }
    __device__ __forceinline__ Vec<E> values() const
    {
        Vec<E> r;
#pragma unroll
        for (int e = 0; e < E; e += 2) bf_pair(v[e / 2], r.v[e], r.v[e + 1]);
        return r;
    }
};
// f(row, values) for rows n of D values from `in`: full batches, then one by one.
template <int D, typename T, typename F>
__device__ __forceinline__ void each_row(const T *in, int n, F f)
{
    constexpr int E = D / 32, B = Raw<E, T>::kBatch;
    int i = 0;
#pragma unroll 1
    for (; i + B <= n; i += B) {
        Raw<E, T> x[B];
#pragma unroll
        for (int u = 0; u < B; ++u) x[u].load(in + (i + u) * D);
#pragma unroll
        for (int u = 0; u < B; ++u) f(i + u, x[u].values());
    }
#pragma unroll 1
    for (; i < n; ++i) {
        Raw<E, T> x;
        x.load(in + i * D);
        f(i, x.values());
    }
}
__device__ __forceinline__ uint32_t bf_pack(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <int E>
__device__ __forceinline__ void store_vec(float *p, const Vec<E> &x)
{
    if constexpr (E == 4) *reinterpret_cast<float4 *>(p) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
    else *reinterpret_cast<float2 *>(p) = make_float2(x.v[0], x.v[1]);
}
template <int E>
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const Vec<E> &x)
{
    if constexpr (E == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(bf_pack(x.v[0], x.v[1]), bf_pack(x.v[2], x.v[3]));
    else *reinterpret_cast<uint32_t *>(p) = bf_pack(x.v[0], x.v[1]);
}

// v (m + lo) rounded once (the product's low part is off by far less than a step).
__device__ __forceinline__ float scaled(uint32_t v, float m, float lo)
{
    const float hi = __uint2float_rz(v), rest = __uint2float_rn(v - __float2uint_rz(hi));      // both exact
    return __fmaf_rn(hi, m, __fmaf_rn(hi, lo, rest * m));
}
// sin and cos of x / 2^64 turns times m + lo, rounded to fp32 correctly in 997 of
// 1000 cases, else a step off: keys come out as from angles in 64 bits, and hardly a
// code next to a border falls to its other side.  (sincospif of a rounded angle is
// 4 us faster in an append of 110 us, and a step off half the time.)  The nearest
// quarter turn is exact; the rest, t eighths of a turn (at most 1), goes through the
// Taylor series of sin and cos of (pi / 4) t in 32-bit fixed point, each coefficient
// (pi / 4)^n / n! 2^32, the sine from a t that is shifted to its first bit.
__device__ __forceinline__ void turn_of(unsigned long long x, float scale, float scale_lo, float &sn, float &cs)
{
    const uint32_t k = static_cast<uint32_t>((x + (1ull << 61)) >> 62);
    const long long r = static_cast<long long>(x - (static_cast<unsigned long long>(k) << 62));
    const unsigned long long m = r < 0 ? 0ull - static_cast<unsigned long long>(r) : static_cast<unsigned long long>(r);
    const uint32_t t = static_cast<uint32_t>((m - (m >> 61)) >> 29), z = __umulhi(t, t);
    uint32_t p = 1346u - __umulhi(8u, z);
    p = 157094u - __umulhi(p, z);
    p = 10696163u - __umulhi(p, z);
    p = 346799334u - __umulhi(p, z);
    p = 3373259426u - __umulhi(p, z);
    const int n = __clzll(static_cast<long long>(m | 1ull));
    const uint32_t first = static_cast<uint32_t>((m << n) >> 32);
    float s = scaled(__umulhi(first, p), scale, scale_lo) * __uint_as_float(static_cast<uint32_t>(98 - n) << 23);      // 2^(-29 - n)
    if (r < 0) s = -s;
    uint32_t q = 15423u - __umulhi(106u, z);
    q = 1400124u - __umulhi(q, z);
    q = 68093890u - __umulhi(q, z);
    q = 1324675879u - __umulhi(q, z);
    const float c = scaled(~__umulhi(z, q), scale, scale_lo) * 2.3283064365386963e-10f;
    sn = __uint_as_float(__float_as_uint(k & 1 ? c : s) ^ (k & 2) << 30);
    cs = __uint_as_float(__float_as_uint(k & 1 ? s : c) ^ ((k + 1) & 2) << 30);
}

// This lane's part of a token's rotation: y[e] = c[e] x[e] + s[e] partner[e].
template <int E>
struct Turn {
    float c[E], s[E];
    int from;             // lane of the partner (HALF), own lane otherwise
    bool half, any;
};
// Lane l takes the sines of pairs A l .. A l + A - 1 (A = E / 2: two for 128
// values), which are its own in the interleaved layout; in halves a lane's E
// pairs come from two (one) other lanes.
template <int E>
__device__ __forceinline__ Turn<E> make_turn(const Rope &R, int pos, int lane, bool inverse)
{
    constexpr int A = E / 2;
    Turn<E> t;
    t.half = R.layout == NQ_ROPE_HALF;
    const int e0 = lane * E, hr = R.rot / 2;
    t.any = e0 < R.rot;
    const bool first = e0 < hr;
    t.from = !t.half || !t.any ? lane : first ? lane + hr / E : lane - hr / E;
    float cs[A], sn[A];
#pragma unroll
    for (int k = 0; k < A; ++k) {
        const int i = A * lane + k;
        const unsigned long long x = static_cast<unsigned long long>(static_cast<long long>(pos)) * (i < hr ? R.rates[i] : 0ull);
        turn_of(x, R.mscale, R.mscale_lo, sn[k], cs[k]);
        if (inverse) sn[k] = -sn[k];
    }
    const int i0 = t.any && !first ? e0 - hr : e0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int src = (i0 + e) / A & 31;
        const float hc = __shfl_sync(0xffffffffu, cs[e % A], src), hs = __shfl_sync(0xffffffffu, sn[e % A], src);
        const float c = t.half ? hc : cs[e / 2], q = t.half ? hs : sn[e / 2];
        t.c[e] = t.any ? c : 1.0f;
        t.s[e] = !t.any ? 0.0f : (t.half ? first : (e & 1) == 0) ? -q : q;
    }
    return t;
}
// Every lane of the warp takes part.
template <int E>
__device__ __forceinline__ Vec<E> turn(const Turn<E> &t, const Vec<E> &x)
{
    Vec<E> y, q;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float p = t.half ? __shfl_sync(0xffffffffu, x.v[e], t.from) : x.v[e ^ 1];
        q.v[e] = p;
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        // both products rounded, as the formula reads: the codes of a key do not depend on how it is evaluated
        const unsigned long long zero = f2_pack(0.0f, 0.0f);
        const float2 z = f2_unpack(f2_add(f2_fma(f2_pack(t.c[e], t.c[e + 1]), f2_pack(x.v[e], x.v[e + 1]), zero),
                                          f2_fma(f2_pack(t.s[e], t.s[e + 1]), f2_pack(q.v[e], q.v[e + 1]), zero)));
        y.v[e] = t.any ? z.x : x.v[e];         // also where the partner, unused, is not finite
        y.v[e + 1] = t.any ? z.y : x.v[e + 1];
    }
    return y;
}

// ---------------------------------------------------------------- rope
template <int D, typename TI, typename TO>
__global__ void __launch_bounds__(kWarps * 32)
rope_kernel(Rope R, const TI *x, long long xs, const int32_t *__restrict__ pos, int T, int H, int per, int chunks,
            bool inverse, TO *out, long long os)
{
    constexpr int E = D / 32;
    const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long t = w / chunks;
    if (t >= T) return;
    const int h0 = static_cast<int>(w % chunks) * per, h1 = min(h0 + per, H);
    const TI *in = x + t * xs + lane * E;
    TO *to = out + t * os + lane * E;
    const Turn<E> tn = make_turn<E>(R, pos[t], lane, inverse);
    each_row<D>(in + h0 * D, h1 - h0, [&](int i, const Vec<E> &v) { store_vec<E>(to + (h0 + i) * D, turn<E>(tn, v)); });
}

// ---------------------------------------------------------------- append
struct Row {              // where a token's row lies
    uint8_t *page;        // record of head 0
    int r;                // row within the page
    bool ok;
};
__device__ __forceinline__ Row row_of(const Pool &p, const Map &m, int s, int pos, unsigned int *status, bool report)
{
    Row w{nullptr, 0, false};
    if (s < 0 || s >= m.S || pos < 0) {
        if (report) set_status(status, NQ_DEV_BAD_PAGE);
        return w;
    }
    const int j = pos / m.P;
    if (j >= m.W) {
        if (report) set_status(status, NQ_DEV_SEQ_FULL);
        return w;
    }
    const int id = m.table[static_cast<size_t>(s) * m.W + j];
    if (id < 0 || id >= p.N) {
        if (report) set_status(status, NQ_DEV_BAD_PAGE);
        return w;
    }
    w.page = p.data + static_cast<size_t>(id) * p.H * p.rec;
    w.r = pos % m.P;
    w.ok = true;
    return w;
}

// nested_quantise's codes of two values, given rs = 1 / s rounded: bytes
// 16 (q4 + 8) + r + 8.  The quotient is the correctly rounded one (Markstein: q +
// (w - q s) / s in fused operations, s having 11 significant bits) wherever it
// is not far below the codes' resolution.  It is held within [-8.49, 7.49], which
// changes no code (beyond, q4 and r are at their ends) and makes q4 = rint(x)
// need no clamp; rounding to whole numbers is adding 1.5 2^23.
__device__ __forceinline__ void codes_of(float w0, float w1, float s, float rs, uint32_t &c0, uint32_t &c1)
{
    const auto both = [](float x) { return f2_pack(x, x); };
    const unsigned long long w = f2_pack(w0, w1), magic = both(12582912.0f), less = both(-12582912.0f), rr = both(rs);
    const unsigned long long q = f2_fma(w, rr, both(0.0f));
    float2 x = f2_unpack(f2_fma(f2_fma(q, both(-s), w), rr, q));
    x.x = fminf(fmaxf(x.x, -8.49f), 7.49f);
    x.y = fminf(fmaxf(x.y, -8.49f), 7.49f);
    const unsigned long long xv = f2_pack(x.x, x.y), a = f2_add(f2_add(xv, magic), less);
    float2 b = f2_unpack(f2_add(f2_fma(f2_sub(xv, a), both(16.0f), magic), less));
    const unsigned long long bv = f2_pack(fminf(b.x, 7.0f), fminf(b.y, 7.0f));
    const float2 c = f2_unpack(f2_fma(a, both(16.0f), f2_add(bv, both(8388744.0f))));    // 2^23 + 136 + 16 q4 + r: exact
    c0 = __float_as_uint(c.x);
    c1 = __float_as_uint(c.y);
}

// Where a lane's part of a K (v = 0) or V (v = 1) row of head 0 lies; the other
// heads' follow p.rec bytes apart.
template <int D, int NG>
struct Place {
    uint8_t *base;
    int resid, scale;     // from base
    __device__ __forceinline__ Place(const Pool &p, const Row &w, int v, int lane)
    {
        constexpr int E = D / 32, RB = D / 2;
        const int blk = w.r >> 4, r16 = w.r & 15;
        if constexpr (NG == 0) {
            base = w.page + blk * p.base_block + v * 32 * D + 2 * bf_off(D, r16, lane * E);
            resid = scale = 0;
        } else {
            const int at = v * 16 * RB + nib_off(RB, r16, lane * E / 2);
            base = w.page + blk * p.base_block + at;
            resid = static_cast<int>(p.resid_off) + blk * (16 * D) - blk * static_cast<int>(p.base_block);
            scale = 32 * RB + v * 32 * NG + (r16 * NG + lane * NG / 32) * 2 - at;
        }
    }
};

// The larger one; NaN where either is NaN.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// One row, quantised in groups of D / NG; true where it is not finite: its group is
// then zeros, so that every reader of the cache sees the same.
template <int D, int NG>
__device__ __forceinline__ bool store_nested(const Place<D, NG> &at, size_t off, const Vec<D / 32> &x, int lane)
{
    constexpr int E = D / 32;
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) amax = max_nan(amax, fabsf(x.v[e]));
#pragma unroll
    for (int o = 16 / NG; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // absmax / 7, correctly rounded as in codes_of
    const float q7 = amax * 0.142857142857142857f;
    __half sh = __float2half_rn(__fmaf_rn(__fmaf_rn(-q7, 7.0f, amax), 0.142857142857142857f, q7));
    const bool bad = !(__half2float(sh) <= 65504.0f);            // a value that is not finite, or past 7 times fp16's largest
    if (bad) sh = __ushort_as_half(0);
    const float s = __half2float(sh), rs = __frcp_rn(s);
    uint32_t c[E], b, r;
#pragma unroll
    for (int e = 0; e < E; e += 2) codes_of(x.v[e], x.v[e + 1], s, rs, c[e], c[e + 1]);
    uint8_t *to = at.base + off;
    if constexpr (E == 4) {
        const uint32_t lo = __byte_perm(c[0], c[2], 0x0040), hi = __byte_perm(c[1], c[3], 0x0040);   // bytes 0, 1: values 0, 2 and 1, 3
        b = (lo >> 4 & 0x0F0Fu) | (hi & 0xF0F0u);
        r = (lo & 0x0F0Fu) | (hi << 4 & 0xF0F0u);
        b = s == 0.0f ? 0x8888u : b;                             // zeros
        r = s == 0.0f ? 0x8888u : r;
        *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(b);
        *reinterpret_cast<uint16_t *>(to + at.resid) = static_cast<uint16_t>(r);
    } else {
        b = (c[0] >> 4 & 0x0Fu) | (c[1] & 0xF0u);
        r = (c[0] & 0x0Fu) | (c[1] << 4 & 0xF0u);
        to[0] = static_cast<uint8_t>(s == 0.0f ? 0x88u : b);
        to[at.resid] = static_cast<uint8_t>(s == 0.0f ? 0x88u : r);
    }
    if (lane % (32 / NG) == 0) *reinterpret_cast<__half *>(to + at.scale) = sh;
    return bad;
}

// NG = 0: BF16.  Rows of a token in the order q heads, k heads, v heads; a warp
// takes a run of them.
template <int D, int NG, typename TI>
__global__ void __launch_bounds__(kWarps * 32)
append_kernel(Pool p, Map m, Rope R, bool rope, const TI *__restrict__ q, const TI *__restrict__ k,
              const TI *__restrict__ v, long long stride, const int32_t *__restrict__ seqs,
              const int32_t *__restrict__ pos, const int32_t *__restrict__ angle, int T, int Hq, int per, int chunks,
              __nv_bfloat16 *__restrict__ q_out, unsigned int *status)
{
    constexpr int E = D / 32;
    const long long wi = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long t = wi / chunks;
    if (t >= T) return;
    const int H = p.H, h0 = static_cast<int>(wi - t * chunks) * per, h1 = min(h0 + per, Hq + 2 * H);
    const int ps = pos[t];
    const Row w = row_of(p, m, seqs[t], ps, status, lane == 0 && h1 > Hq);
    Turn<E> tn{};
    const bool turned = rope && h0 < Hq + H;
    if (turned) tn = make_turn<E>(R, angle[t], lane, false);
    const long long at = t * stride + lane * E;
    if (h0 < Hq) {
        __nv_bfloat16 *to = q_out + (t * Hq + h0) * D + lane * E;
        each_row<D>(q + at + h0 * D, min(h1, Hq) - h0, [&](int i, const Vec<E> &x) { store_vec<E>(to + i * D, turned ? turn<E>(tn, x) : x); });
    }
    if (!w.ok) return;
    bool bad = false;
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
        const int a = max(h0 - Hq - kv * H, 0), b = min(h1 - Hq - kv * H, H);
        if (a >= b) continue;
        const Place<D, NG> place(p, w, kv, lane);
        const bool tk = turned && kv == 0;
        each_row<D>((kv ? v : k) + at + a * D, b - a, [&](int i, const Vec<E> &x0) {
            const Vec<E> x = tk ? turn<E>(tn, x0) : x0;
            const size_t off = static_cast<size_t>(a + i) * p.rec;
            if constexpr (NG == 0) store_vec<E>(reinterpret_cast<__nv_bfloat16 *>(place.base + off), x);
            else bad |= store_nested<D, NG>(place, off, x, lane);
        });
    }
    if (bad) set_status(status, NQ_DEV_NONFINITE);
}

// ---------------------------------------------------------------- read
// One warp per token and run of heads: their K and V rows.
template <int D, int NG>
__global__ void __launch_bounds__(kWarps * 32)
read_kernel(Pool p, Map m, const int32_t *__restrict__ seqs, const int32_t *__restrict__ pos, int T, int planes, int per,
            int chunks, __nv_bfloat16 *__restrict__ k_out, __nv_bfloat16 *__restrict__ v_out, unsigned int *status)
{
    constexpr int E = D / 32, RB = D / 2, U = 4;
    const unsigned wi = blockIdx.x * kWarps + (threadIdx.x >> 5), t = wi / chunks;
    const int lane = threadIdx.x & 31;
    if (t >= static_cast<unsigned>(T)) return;
    const int h0 = static_cast<int>(wi - t * chunks) * per, h1 = min(h0 + per, p.H);
    const Row w = row_of(p, m, seqs[t], pos[t], status, lane == 0);
    const int blk = w.r >> 4, r16 = w.r & 15;
    const uint8_t *base = w.page + blk * p.base_block, *resid = w.page + p.resid_off + blk * (16 * D);
    const uint32_t at = NG == 0 ? 2 * bf_off(D, r16, lane * E) : nib_off(RB, r16, lane * E / 2);
    const uint32_t sat = 32 * RB + (r16 * NG + lane * NG / 32) * 2;
    for (int h = h0; h < h1; h += U) {        // the loads of U rows of K and of V before the first is used
        uint32_t b[U][2][2];
        unsigned short sc[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u >= h1) continue;
            if (!w.ok) {                      // zeros
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    b[u][v][0] = b[u][v][1] = NG == 0 ? 0u : 0x8888u;
                    sc[u][v] = 0;
                }
                continue;
            }
            const size_t rec = static_cast<size_t>(h + u) * p.rec;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if constexpr (NG == 0) {
                    const uint8_t *src = base + rec + v * 32 * D + at;
                    if constexpr (E == 4) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(src);
                        b[u][v][0] = x.x;
                        b[u][v][1] = x.y;
                    } else {
                        b[u][v][0] = *reinterpret_cast<const uint32_t *>(src);
                    }
                } else {
                    sc[u][v] = *reinterpret_cast<const unsigned short *>(base + rec + sat + v * 32 * NG);
                    if constexpr (E == 4) {
                        b[u][v][0] = *reinterpret_cast<const uint16_t *>(base + rec + v * 16 * RB + at);
                        b[u][v][1] = planes == 2 ? *reinterpret_cast<const uint16_t *>(resid + rec + v * 16 * RB + at) : 0x8888u;
                    } else {
                        b[u][v][0] = base[rec + v * 16 * RB + at];
                        b[u][v][1] = planes == 2 ? resid[rec + v * 16 * RB + at] : 0x8888u;
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u >= h1) continue;
            const size_t to = (static_cast<size_t>(t) * p.H + h + u) * D + lane * E;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                Vec<E> x;
                if constexpr (NG == 0) {
                    bf_pair(b[u][v][0], x.v[0], x.v[1]);
                    if constexpr (E == 4) bf_pair(b[u][v][1], x.v[2], x.v[3]);
                } else {
                    const float s = __half2float(__ushort_as_half(sc[u][v])) * 0.0625f;
                    // bytes 16 (q4 + 8) + r + 8 of the even and the odd values, each then the
                    // low byte of the number 2^23 + byte
                    const uint32_t lo = (b[u][v][0] << 4 & 0xF0F0u) | (b[u][v][1] & 0x0F0Fu);
                    const uint32_t hi = (b[u][v][0] & 0xF0F0u) | (b[u][v][1] >> 4 & 0x0F0Fu);
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float c0 = __uint_as_float(__byte_perm(lo, 0x4B000000u, 0x7550 | (e >> 1)));
                        const float c1 = __uint_as_float(__byte_perm(hi, 0x4B000000u, 0x7550 | (e >> 1)));
                        x.v[e] = s * (c0 - 8388744.0f);
                        x.v[e + 1] = s * (c1 - 8388744.0f);
                    }
                }
                store_vec<E>((v ? v_out : k_out) + to, x);
            }
        }
    }
}

// ---------------------------------------------------------------- host side
nq_status rope_of(const nq_rope_plan *r, int head_dim, Rope &out)
{
    if (!r || !r->rates || !(r->layout == NQ_ROPE_HALF || r->layout == NQ_ROPE_INTERLEAVED)) return NQ_ERR_ARG;
    if (r->rot_dim < 8 || r->rot_dim % 8 != 0 || r->rot_dim > head_dim) return NQ_ERR_SHAPE;
    if (!aligned16(r->rates)) return NQ_ERR_ALIGN;
    out = Rope{r->rot_dim, r->layout, r->mscale, r->mscale_lo, reinterpret_cast<const unsigned long long *>(r->rates)};
    return NQ_OK;
}
// Heads per warp: up to 48 for prompts, where the sines of a token serve them all,
// and down to one, so that a small call spreads over the machine (16 warps per SM).
// Append of 8191 tokens, 96 heads: 109 us with two runs, 119 with three (of q, k
// and v rows, which cost unlike), 132 with twelve of 8.  Of 144 tokens, 48 heads:
// 4.9 us; 8.5 in runs of 32, 6.5 with twice the warps.  Rotating 16384 tokens of
// 32 heads: 44 us whole, 51 in runs of 8.
int heads_per_warp(long long T, int heads)
{
    int chunks = (heads + 47) / 48;
    while (chunks < heads && T * chunks < 16ll * sm_count()) chunks *= 2;
    return (heads + chunks - 1) / chunks;
}

template <int D, typename TI, typename TO>
void launch_rope(const Rope &R, const void *x, long long xs, const int32_t *pos, int T, int H, bool inverse, void *out,
                 long long os, cudaStream_t s)
{
    const int per = heads_per_warp(T, H), chunks = (H + per - 1) / per;
    const long long warps = static_cast<long long>(T) * chunks;
    rope_kernel<D, TI, TO><<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(
        R, static_cast<const TI *>(x), xs, pos, T, H, per, chunks, inverse, static_cast<TO *>(out), os);
}
template <int D>
void launch_rope_t(const Rope &R, const void *x, int xt, long long xs, const int32_t *pos, int T, int H, bool inverse,
                   void *out, int ot, long long os, cudaStream_t s)
{
    using B = __nv_bfloat16;
    if (xt == NQ_F32) {
        if (ot == NQ_F32) launch_rope<D, float, float>(R, x, xs, pos, T, H, inverse, out, os, s);
        else launch_rope<D, float, B>(R, x, xs, pos, T, H, inverse, out, os, s);
    } else {
        if (ot == NQ_F32) launch_rope<D, B, float>(R, x, xs, pos, T, H, inverse, out, os, s);
        else launch_rope<D, B, B>(R, x, xs, pos, T, H, inverse, out, os, s);
    }
}

template <int D, int NG, typename TI>
void launch_append(const Pool &p, const Map &m, const Rope &R, bool rope, const void *q, const void *k, const void *v,
                   long long stride, const int32_t *seqs, const int32_t *pos, const int32_t *angle, int T, int Hq, void *q_out,
                   unsigned int *status, cudaStream_t s)
{
    const int all = Hq + 2 * p.H, per = heads_per_warp(T, all), chunks = (all + per - 1) / per;
    const long long warps = static_cast<long long>(T) * chunks;
    append_kernel<D, NG, TI><<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(
        p, m, R, rope, static_cast<const TI *>(q), static_cast<const TI *>(k), static_cast<const TI *>(v), stride, seqs,
        pos, angle, T, Hq, per, chunks, static_cast<__nv_bfloat16 *>(q_out), status);
}

}  // namespace
}  // namespace nq

extern "C" nq_status nq_rope_mscale(int scaling, double factor, float *mscale, float *mscale_lo)
{
    if (!mscale || !mscale_lo || scaling < NQ_ROPE_NONE || scaling > NQ_ROPE_PARTS) return NQ_ERR_ARG;
    if (scaling != NQ_ROPE_NONE && !(factor >= 1.0 && std::isfinite(factor))) return NQ_ERR_ARG;
    const double m = scaling == NQ_ROPE_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
    *mscale = static_cast<float>(m);
    *mscale_lo = static_cast<float>(m - *mscale);
    return NQ_OK;
}

extern "C" nq_status nq_rope_rates(int rot_dim, double theta, int scaling, double factor, int old_len, uint64_t *rates,
                                   float *mscale)
{
    float m, m_lo;
    if (!rates || !mscale || !(theta > 1.0) || !std::isfinite(theta)) return NQ_ERR_ARG;
    if (nq_rope_mscale(scaling, factor, &m, &m_lo) != NQ_OK) return NQ_ERR_ARG;
    if (scaling == NQ_ROPE_PARTS && old_len < 1) return NQ_ERR_ARG;
    if (rot_dim < 8 || rot_dim % 8 != 0 || rot_dim > 128) return NQ_ERR_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == NQ_ROPE_NTK) theta *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    *mscale = m;
    for (int i = 0; i < rot_dim / 2; ++i) {
        double w = std::pow(theta, -2.0 * i / rot_dim);
        if (scaling == NQ_ROPE_LINEAR) w /= factor;
        if (scaling == NQ_ROPE_PARTS) {
            double keep = (old_len * w / two_pi - 1.0) / 31.0;
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            w = w * keep + w / factor * (1.0 - keep);
        }
        // w <= 1, so the rate is below 2^64 / 6
        rates[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(w / two_pi, 64)));
    }
    return NQ_OK;
}

extern "C" nq_status nq_rope(const nq_rope_plan *rope, const void *x, int x_dtype, int64_t x_stride, const int32_t *pos,
                             int T, int heads, int head_dim, int inverse, void *out, int out_dtype, int64_t out_stride,
                             cudaStream_t stream)
{
    if (!x || !pos || !out || T < 1 || heads < 1) return NQ_ERR_ARG;
    if (!(x_dtype == NQ_F32 || x_dtype == NQ_BF16) || !(out_dtype == NQ_F32 || out_dtype == NQ_BF16)) return NQ_ERR_ARG;
    if (!(head_dim == 64 || head_dim == 128) || heads > 65536) return NQ_ERR_SHAPE;
    const int64_t row = static_cast<int64_t>(heads) * head_dim;
    if (x_stride < row || out_stride < row || x_stride % 8 != 0 || out_stride % 8 != 0) return NQ_ERR_SHAPE;
    nq::Rope R;
    const nq_status st = nq::rope_of(rope, head_dim, R);
    if (st != NQ_OK) return st;
    if (!nq::aligned16(x) || !nq::aligned16(out) || !nq::aligned4(pos)) return NQ_ERR_ALIGN;
    if (x == out && (x_dtype != out_dtype || x_stride != out_stride)) return NQ_ERR_ARG;
    if (static_cast<double>(T) * heads / nq::kWarps > 2147483000.0) return NQ_ERR_SHAPE;
    if (head_dim == 128)
        nq::launch_rope_t<128>(R, x, x_dtype, x_stride, pos, T, heads, inverse != 0, out, out_dtype, out_stride, stream);
    else
        nq::launch_rope_t<64>(R, x, x_dtype, x_stride, pos, T, heads, inverse != 0, out, out_dtype, out_stride, stream);
    return nq::cuda_status(cudaGetLastError());
}

extern "C" nq_status nq_page_append_at(const nq_page_pool *pool, int layer, const nq_page_map *map,
                                       const nq_rope_plan *rope, const void *q, const void *k, const void *v, int dtype,
                                       int64_t stride, const int32_t *seqs, const int32_t *pos, const int32_t *angle, int T,
                                       int heads_q, uint16_t *q_out, cudaStream_t stream)
{
    nq::Pool p;
    nq::Map m;
    nq_status st = nq::pool_map_of(pool, map, p, m, false);
    if (st != NQ_OK) return st;
    if (layer < 0 || layer >= pool->layers || !k || !v || !seqs || !pos || !angle || T < 1) return NQ_ERR_ARG;
    if (!(dtype == NQ_F32 || dtype == NQ_BF16)) return NQ_ERR_ARG;
    if (q ? (heads_q < 1 || !q_out) : (heads_q != 0 || q_out != nullptr)) return NQ_ERR_ARG;
    if (heads_q > 65536) return NQ_ERR_SHAPE;
    const int64_t row = static_cast<int64_t>(heads_q > p.H ? heads_q : p.H) * p.D;
    if (stride < row || stride % 8 != 0) return NQ_ERR_SHAPE;
    nq::Rope R{};
    if (rope) {
        st = nq::rope_of(rope, p.D, R);
        if (st != NQ_OK) return st;
    }
    if (!nq::aligned16(k) || !nq::aligned16(v) || !nq::aligned16(q) || !nq::aligned16(q_out) || !nq::aligned4(seqs) ||
        !nq::aligned4(pos) || !nq::aligned4(angle))
        return NQ_ERR_ALIGN;
    if (static_cast<double>(T) * (heads_q + 2.0 * p.H) / nq::kWarps > 2147483000.0) return NQ_ERR_SHAPE;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    p.data += static_cast<size_t>(layer) * p.layer_bytes;
    auto go = [&](auto d, auto ng) {
        constexpr int D = decltype(d)::value, NG = decltype(ng)::value;
        if (dtype == NQ_F32)
            nq::launch_append<D, NG, float>(p, m, R, rope != nullptr, q, k, v, stride, seqs, pos, angle, T, heads_q, q_out, status, stream);
        else
            nq::launch_append<D, NG, __nv_bfloat16>(p, m, R, rope != nullptr, q, k, v, stride, seqs, pos, angle, T, heads_q, q_out, status, stream);
    };
    using std::integral_constant;
    const integral_constant<int, 64> d64;
    const integral_constant<int, 128> d128;
    const integral_constant<int, 0> bf;
    const integral_constant<int, 1> g1;
    const integral_constant<int, 2> g2;
    if (p.D == 64) p.NG == 0 ? go(d64, bf) : go(d64, g1);
    else p.NG == 0 ? go(d128, bf) : p.NG == 1 ? go(d128, g1) : go(d128, g2);
    return nq::cuda_status(cudaGetLastError());
}

extern "C" nq_status nq_page_append(const nq_page_pool *pool, int layer, const nq_page_map *map,
                                    const nq_rope_plan *rope, const void *q, const void *k, const void *v, int dtype,
                                    int64_t stride, const int32_t *seqs, const int32_t *pos, int T, int heads_q,
                                    uint16_t *q_out, cudaStream_t stream)
{
    return nq_page_append_at(pool, layer, map, rope, q, k, v, dtype, stride, seqs, pos, pos, T, heads_q, q_out, stream);
}

extern "C" nq_status nq_page_read(const nq_page_pool *pool, int layer, const nq_page_map *map, const int32_t *seqs,
                                  const int32_t *pos, int T, int planes, uint16_t *k_out, uint16_t *v_out,
                                  cudaStream_t stream)
{
    nq::Pool p;
    nq::Map m;
    const nq_status st = nq::pool_map_of(pool, map, p, m, false);
    if (st != NQ_OK) return st;
    if (layer < 0 || layer >= pool->layers || !seqs || !pos || !k_out || !v_out || T < 1 || (planes != 1 && planes != 2))
        return NQ_ERR_ARG;
    if (!nq::aligned16(k_out) || !nq::aligned16(v_out) || !nq::aligned4(seqs) || !nq::aligned4(pos)) return NQ_ERR_ALIGN;
    const long long warps = static_cast<long long>(T) * p.H;
    if (warps > 4294960000ll) return NQ_ERR_SHAPE;
    unsigned int *status = nq::device_status_ptr();
    if (!status) return NQ_ERR_CUDA;
    p.data += static_cast<size_t>(layer) * p.layer_bytes;
    const int per = nq::heads_per_warp(T, p.H), chunks = (p.H + per - 1) / per;
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(T) * chunks + nq::kWarps - 1) / nq::kWarps);
    auto *ko = reinterpret_cast<__nv_bfloat16 *>(k_out), *vo = reinterpret_cast<__nv_bfloat16 *>(v_out);
    auto go = [&](auto *kernel) { kernel<<<grid, nq::kWarps * 32, 0, stream>>>(p, m, seqs, pos, T, planes, per, chunks, ko, vo, status); };
    if (p.D == 64) go(p.NG == 0 ? nq::read_kernel<64, 0> : nq::read_kernel<64, 1>);
    else go(p.NG == 0 ? nq::read_kernel<128, 0> : p.NG == 1 ? nq::read_kernel<128, 1> : nq::read_kernel<128, 2>);
    return nq::cuda_status(cudaGetLastError());
}
