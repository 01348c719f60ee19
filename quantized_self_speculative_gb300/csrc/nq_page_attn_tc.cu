// nq_page_attn_tc.cu -- attention over nested pages for many query vectors per
// kv head (from 25 on, heads of 64 from 33: a verify pass with grouped queries), on
// the 5th-generation tensor cores.
//
// With many query vectors the products and the decoding bound the time, not
// HBM.  Here a row of the tensor cores is a query vector (up to 128 per tile):
// S = Q K^T and O += P V with Q, P and both accumulators in tensor memory, and
// K and V^T decoded once per step of 64 cache rows into shared memory as signed
// fp16 codes (exact; the scales of K multiply S, those of V multiply P).  Both
// are then K-major operands, so V is transposed on the way: eight rows of eight
// dimensions at a time by movmatrix.  A softmax row belongs to one thread: no
// shuffles, one load of scores and one store of P per step.
//
// Warp roles, handing on through mbarriers (all waits bounded):
//   0-3   softmax: lane quarter w of tensor memory; also Q in, O out
//   4-11  decode: stage -> K, V^T, scales (four buffers: up to three steps ahead)
//   12    issues the MMAs: S of the next step before P V of this one
//   13    feeds the ring of raw blocks
// O is only rescaled when a row's maximum has grown by 2^12, which waits for
// the product before.  One CTA per SM (512 columns of tensor memory), the same
// runs, partial states and join as the other kernels.
//
// Measured (GB300): 16 sequences of 301..4099 rows, 8 kv heads of 128, 9 rows x 4
// heads = 36 query vectors, 8-bit view: 65 us for 79 MB (12 us at the copy rate).
// Per step of 64 rows the softmax warps take some 1700 cycles, the decoders 1300,
// the tensor pipe 512: bound by the softmax chain (load S, scale, maximum, exp2,
// store P), and by the ends of segments, where the pipeline drains.
#include <atomic>

#include "nq_page_attn.cuh"
#include "nq_tcgen.cuh"

namespace nq {
namespace {

constexpr int kSoftWarps = 4, kDecodeWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kDecodeWarps, kFeedWarp = kMmaWarp + 1;
constexpr int kThreads = (kFeedWarp + 1) * 32;
constexpr int kMinRun = 2;              // steps per CTA
constexpr int kKeys = 64;               // cache rows per step
constexpr int kBufs = 4;                // decoded steps
constexpr int kTmem = 512;              // columns: Q at 0 (D / 2), S at 64 (two of 64), P at 192 (two of 32), O at 256 (D)
constexpr uint32_t kColS = 64, kColP = 192, kColO = 256;

template <int FMT, int D>
struct Tc {
    static constexpr int BASE = block_base(FMT, D, 1), RESID = block_resid(FMT, D);
    static constexpr int BLKS = kKeys / 16, STAGE = BLKS * (BASE + RESID);
    static constexpr int K_BYTES = kKeys * D * 2, V_BYTES = D * kKeys * 2;
    static constexpr int BUF = K_BYTES + V_BYTES;                // one step, both operands in 1024-byte groups
    static constexpr int SCALES = 3 * kKeys * 4;                 // K's, V's, log2 of V's
    static constexpr int STAGES = 4;
    static constexpr int SMEM = kBufs * (BUF + SCALES) + STAGES * STAGE;
};

// Barriers by number.
constexpr int kRawFull = 0, kRawEmpty = 4, kKvFull = 8, kKvEmpty = 12, kPvDone = 16, kSFull = 18, kPFull = 20, kQFull = 22, kDrain = 23, kBars = 24;

template <int FMT, int D, bool X>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ AttnArgs A)
{
    using Q = Tc<FMT, D>;
    constexpr int SR = kKeys, BLKS = Q::BLKS, RB = D / 2;
    static_assert(Q::STAGES == 4 && kBufs == 4, "barrier numbers");
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ __align__(8) unsigned long long bars[kBars];
    __shared__ uint32_t gone_of[Q::STAGES], gone_decoded[kBufs];                 // blocks that are not there
    __shared__ int abort_flag, keep_tmem;
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int segs = A.p.H * A.QT;
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](int i) { return bar0 + 8u * i; };
    if (threadIdx.x == 0) {
        abort_flag = keep_tmem = 0;
        A.info[blockIdx.x] = make_int4(-1, 0, 0, 0);             // until the CTA has left a part for the join
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kRawFull + i), 1);
            mbar_init(bar(kRawEmpty + i), kDecodeWarps);
            mbar_init(bar(kKvFull + i), kDecodeWarps);
            mbar_init(bar(kKvEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kPvDone + i), 1);
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kPFull + i), kSoftWarps);
        }
        mbar_init(bar(kQFull), kSoftWarps);
        mbar_init(bar(kDrain), 32);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const Run run = find_run<SR, kThreads, D>(A, segs, kMinRun);
    if (run.f0 >= run.f1) return;
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    unsigned char *scales = sm + kBufs * Q::BUF, *ring = scales + kBufs * Q::SCALES;
    auto wait = [&](int i, int phase) { return mbar_wait_fast(bar(i), static_cast<uint32_t>(phase) & 1u, &abort_flag, A.status, A.wait_ns); };
    const int steps = run.f1 - run.f0;
    Walk<SR> use;
    use.open(A, run.b, run.base, run.f0, run.f1);

    if (warp == kFeedWarp) {
        // ================================================= raw blocks into the ring
        Feed<FMT, D, 1, BLKS, 1> feed;
        feed.start(A, use, segs, run.f0, smem_u32(ring), bar(kRawFull));
        int i = 0;
        for (; i < steps && feed.left > 0; ++i) {
            const int st = i % Q::STAGES;
            if (!__all_sync(0xffffffffu, wait(kRawEmpty + st, (i / Q::STAGES & 1) ^ 1))) break;
            feed.issue(A, segs, st, [&](uint32_t out) { gone_of[st] = out; });
        }
        // every copy issued has landed before the CTA may exit
        volatile int never = 0;
        for (int k = max(0, i - Q::STAGES); k < i; ++k) mbar_wait(bar(kRawFull + k % Q::STAGES), k / Q::STAGES & 1, &never, A.status, A.wait_ns);
    } else if (warp >= kSoftWarps && warp < kMmaWarp) {
        // ================================================= decode
        const int dw = warp - kSoftWarps, g = lane >> 2, t = lane & 3;
        for (int i = 0; i < steps; ++i) {
            const int st = i % Q::STAGES, b = i % kBufs;
            if (!__all_sync(0xffffffffu, wait(kRawFull + st, i / Q::STAGES & 1) && wait(kKvEmpty + b, (i / kBufs & 1) ^ 1))) break;
            const unsigned char *sp = ring + st * Q::STAGE;
            unsigned char *kt = sm + b * Q::BUF, *vt = kt + Q::K_BYTES;
            // ---- K: thread = (row, 16-byte chunk of nibbles): four words of eight values, in
            // the order 0 4 1 5 2 6 3 7 that the masks give (Q's columns follow it)
            {
                constexpr int CH = RB / 16;                      // 4 (D = 128) or 2
                const int e = dw * 32 + lane;
                if (e < kKeys * CH) {
                    const int r = e / CH, c = e % CH, at = nib_off(RB, r & 15, 16 * c);
                    uint4 x = *reinterpret_cast<const uint4 *>(sp + (r >> 4) * Q::BASE + at), y = make_uint4(0, 0, 0, 0);
                    if constexpr (FMT == kKv8) y = *reinterpret_cast<const uint4 *>(sp + BLKS * Q::BASE + (r >> 4) * Q::RESID + at);
                    // chunks of the upper 64 dimensions in another order: then eight lanes write to eight banks
                    const bool swap = c >= 2;
                    const uint32_t xw[4] = {swap ? x.z : x.x, swap ? x.w : x.y, swap ? x.x : x.z, swap ? x.y : x.w};
                    const uint32_t yw[4] = {swap ? y.z : y.x, swap ? y.w : y.y, swap ? y.x : y.z, swap ? y.y : y.w};
                    unsigned char *to = kt + (c >> 1) * (kKeys * 128) + r * 128;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const Codes<FMT> k(xw[w], yw[w]);
                        const int chunk = 4 * (c & 1) + (swap ? w ^ 2 : w);
                        *reinterpret_cast<uint4 *>(to + ((chunk ^ (r & 7)) << 4)) = make_uint4(k.value(0), k.value(1), k.value(2), k.value(3));
                    }
                }
                // ---- scales
                if (e < kKeys) {
                    const __half *sc = reinterpret_cast<const __half *>(sp + (e >> 4) * Q::BASE + 32 * RB);
                    float *f = reinterpret_cast<float *>(scales + b * Q::SCALES);
                    // a scale that is not finite, or negative, counts as 0: rows past the end may hold anything
                    float sk = __half2float(sc[e & 15]), sv = __half2float(sc[16 + (e & 15)]);
                    sk = sk >= 0.0f && sk <= 65504.0f ? sk : 0.0f;
                    sv = sv >= 0.0f && sv <= 65504.0f ? sv : 0.0f;
                    if (e == 0) gone_decoded[b] = gone_of[st];
                    f[e] = sk;
                    f[kKeys + e] = sv;
                    f[2 * kKeys + e] = lg2(fmaxf(sv, 3.7252902984619140625e-09f));   // a scale of 0 has codes of 0
                }
            }
            // ---- V^T: warp dw takes rows 8 dw .. 8 dw + 7, lane (g, t) chunk t of row g.  Words are turned
            // by t nibbles, so that the eight columns of a transposed block are eight dimensions mod 8
            // and its stores meet no bank twice.
            {
                constexpr int NW = D / 32;                       // words per lane: 4 (D = 128) or 2
                const int r = 8 * dw + g, at = 16 * RB + nib_off(RB, r & 15, NW * 4 * t);
                uint32_t xw[NW], yw[NW];
                const unsigned char *bp = sp + (r >> 4) * Q::BASE + at, *rp = sp + BLKS * Q::BASE + (r >> 4) * Q::RESID + at;
                if constexpr (NW == 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(bp);
                    xw[0] = x.x; xw[1] = x.y; xw[2] = x.z; xw[3] = x.w;
                    if constexpr (FMT == kKv8) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(rp);
                        yw[0] = y.x; yw[1] = y.y; yw[2] = y.z; yw[3] = y.w;
                    }
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(bp);
                    xw[0] = x.x; xw[1] = x.y;
                    if constexpr (FMT == kKv8) {
                        const uint2 y = *reinterpret_cast<const uint2 *>(rp);
                        yw[0] = y.x; yw[1] = y.y;
                    }
                }
                // after the transpose this lane holds rows 2 t, 2 t + 1 of the dimension whose column g was
                const int ts = g >> 1, h = g & 1;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const Codes<FMT> k(__funnelshift_r(xw[w], xw[w], 4 * t), FMT == kKv8 ? __funnelshift_r(yw[w], yw[w], 4 * t) : 0u);
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int d = 8 * NW * ts + 8 * w + ((p + ts + 4 * h) & 7);
                        *reinterpret_cast<uint32_t *>(vt + d * 128 + ((dw ^ (d & 7)) << 4) + 4 * t) = [&] {
                            uint32_t y;
                            asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(k.value(p)));
                            return y;
                        }();
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMAs read, and the next copy writes, through the async proxy
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kKvFull + b));
                mbar_arrive(bar(kRawEmpty + st));
            }
        }
    } else if (warp == kMmaWarp) {
        // ================================================= MMAs
        const uint32_t idesc_s = f16_idesc(128, kKeys), idesc_o = f16_idesc(128, D);
        uint32_t issued_by = 0;
        bool ok = true;
        int issued_s = 0, seg_no = 0;         // S products issued; segments begun
        auto scores = [&](int i, bool first) {                   // S of step i
            bool w = wait(kKvFull + i % kBufs, i / kBufs & 1);
            if (first) w = w && wait(kQFull, seg_no & 1);
            if (!__all_sync(0xffffffffu, w)) return false;
            if (first) ++seg_no;
            tc_fence_after();
            const uint32_t kt = smem_u32(sm + i % kBufs * Q::BUF);
            uint32_t leader;
            if (elect_one(leader)) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma(tmem + kColS + 64 * (i & 1), tmem + 8 * k, sw128_desc(kt + (k >> 2) * (kKeys * 128) + (k & 3) * 32), idesc_s, k != 0);
                tc_commit(bar(kSFull + (i & 1)));
            }
            __syncwarp();
            issued_by |= 1u << leader;
            return true;
        };
        bool first = true;                    // step i begins its segment (part)
        for (int i = 0; i < steps && ok; ++i) {
            const bool last = run.f0 + i + 1 >= use.end;
            if (issued_s == i) {
                ok = scores(i, first);
                ++issued_s;
            }
            if (ok && !last && i + 1 < steps) {
                ok = scores(i + 1, false);
                ++issued_s;
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, wait(kPFull + (i & 1), i >> 1 & 1));
            if (!ok) break;
            tc_fence_after();
            const uint32_t vt = smem_u32(sm + i % kBufs * Q::BUF + Q::K_BYTES);
            uint32_t leader;
            if (elect_one(leader)) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    tc_mma(tmem + kColO, tmem + kColP + 32 * (i & 1) + 8 * k, sw128_desc(vt + k * 32), idesc_o, !first || k != 0);
                tc_commit(bar(kPvDone + (i & 1)));
                tc_commit(bar(kKvEmpty + i % kBufs));
            }
            __syncwarp();
            issued_by |= 1u << leader;
            first = last;
            if (last && i + 1 < steps) use.next(A, segs);
        }
        // every MMA has completed before tensor memory is freed, whatever ended the loop
        if (issued_by) {
            if ((issued_by >> lane) & 1u) tc_commit(bar(kDrain));
            else mbar_arrive(bar(kDrain));
            __syncwarp();
            volatile int never = 0;
            const bool drained = mbar_wait(bar(kDrain), 0, &never, A.status, A.wait_ns);
            if (!__all_sync(0xffffffffu, drained) && lane == 0) keep_tmem = 1;
        }
    } else {
        // ================================================= softmax: thread = query vector
        const int row = warp * 32 + lane;
        const uint32_t tq = tmem + (static_cast<uint32_t>(warp) << 21);          // lanes 32 w ..
        const float cap2 = A.softcap * kLog2e, inv2 = X && A.softcap > 0.0f ? 1.0f / cap2 : 0.0f;
        const unsigned window = A.window > 0 ? A.window : 0x7fffffffu;
        bool fresh = true, active = false;
        int kvh = 0, v0 = 0, nv = 0, own = 0, all_lo = 0, all_hi = 0, m = 0;
        float cq = 0.0f, slope2 = 0.0f, mref = 0.0f, mz = 0.0f, lsum = 0.0f;
        for (int i = 0; i < steps; ++i) {
            if (fresh) {
                // ---- the segment's query rows into tensor memory
                fresh = false;
                kvh = use.seg / A.QT;
                v0 = (use.seg - kvh * A.QT) * A.cols;
                nv = min(A.cols, A.M * A.G - v0);
                active = 32 * warp < nv;
                const bool valid = row < nv;
                m = row_of_vector(A, valid ? v0 + row : v0 + nv - 1);
                const int hq = kvh * A.G + (valid ? v0 + row : v0 + nv - 1) - m * A.G;
                if (active) {
                    const uint4 *qr = reinterpret_cast<const uint4 *>(A.q + (static_cast<long long>(use.b) * A.M + m) * A.q_stride + hq * D);
                    float top = 0.0f;
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 x = qr[c];
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[u] << 16)), fabsf(__uint_as_float(w[u] & 0xFFFF0000u))));
                    }
                    // largest magnitude to [2^10, 2^11) by a power of two
                    const int up = min(137 - static_cast<int>(__float_as_uint(top) >> 23), 120);
                    const float to = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                    cq = fmaxf(A.scale * kLog2e * (FMT == kKv8 ? 0.0625f : 1.0f) * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 1.2e-38f);
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {           // 16 columns: 32 values
                        uint32_t y[16];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint4 x = qr[4 * c + u];
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                            float f[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                f[2 * k] = __uint_as_float(w[k] << 16) * to;
                                f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * to;
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) y[4 * u + k] = pack_h(f[k], f[k + 4]);
                        }
                        tc_st16(tq + 16 * c, y);
                    }
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kQFull));
                own = use.s.hi - A.M + m;
                slope2 = X && A.slopes ? A.slopes[hq] * kLog2e : 0.0f;
                all_hi = use.s.hi - A.M + row_of_vector(A, v0) + 1;
                all_lo = first_seen(A, use.s.hi - A.M + row_of_vector(A, v0 + nv - 1));
                mref = -INFINITY;
                mz = lsum = 0.0f;
            }
            const int b = i & 1, row0 = use.s.lo + (run.f0 + i - use.base) * SR;
            const bool begins = run.f0 + i == max(use.base, run.f0), masked = row0 < all_lo || row0 + SR > all_hi;
            // S is there, and the P of two steps ago has been used
            if (!__all_sync(0xffffffffu, wait(kSFull + b, i >> 1 & 1) && wait(kPvDone + b, (i >> 1 & 1) ^ 1))) break;
            bool gave_up = false;
            if (active) {
                tc_fence_after();
                uint32_t s[64];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc_ld16(tq + kColS + 64 * b + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(s + 16 * c));
                tc_wait_ld();
                const float *f = reinterpret_cast<const float *>(scales + i % kBufs * Q::SCALES);
                const uint32_t gone = gone_decoded[i % kBufs];
                // scores in base 2 (X), or what cq makes scores of; two keys at a time in packed fp32
                const unsigned long long zero2 = f2_pack(0.0f, 0.0f), cq2 = f2_pack(cq, cq);
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(f + j);
                    const float2 x[2] = {f2_unpack(f2_fma(f2_pack(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), f2_pack(k4.x, k4.y), zero2)),
                                   f2_unpack(f2_fma(f2_pack(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), f2_pack(k4.z, k4.w), zero2))};
                    s[j] = __float_as_uint(X ? x[0].x * cq : x[0].x);
                    s[j + 1] = __float_as_uint(X ? x[0].y * cq : x[0].y);
                    s[j + 2] = __float_as_uint(X ? x[1].x * cq : x[1].x);
                    s[j + 3] = __float_as_uint(X ? x[1].y * cq : x[1].y);
                }
                if constexpr (X) {
                    if (A.softcap > 0.0f) {
                        if (masked || gone) {
                            const unsigned d = own - row0;
#pragma unroll
                            for (int j = 0; j < 64; ++j) s[j] = d - j >= window || (gone >> (j >> 4) & 1u) ? 0u : s[j];
                        }
                        cap_all(reinterpret_cast<float(&)[64]>(s), cap2, inv2);
                    }
                    if (A.slopes) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            s[j] = __float_as_uint(fmaf(slope2, static_cast<float>(row0 + j - own), __uint_as_float(s[j])));
                    }
                }
                if (masked || gone) {         // before the window, or (negative) after the query's own row; not there
                    const unsigned d = own - row0;
#pragma unroll
                    for (int j = 0; j < 64; ++j) s[j] = d - j >= window || (gone >> (j >> 4) & 1u) ? 0xFF800000u : s[j];
                }
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};    // with the log2 of V's scales
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 l4 = *reinterpret_cast<const float4 *>(f + 2 * kKeys + j);
                    const unsigned long long x0 = f2_pack(__uint_as_float(s[j]), __uint_as_float(s[j + 1])),
                                             x1 = f2_pack(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
                    const float2 y0 = f2_unpack(X ? f2_add(x0, f2_pack(l4.x, l4.y)) : f2_fma(x0, cq2, f2_pack(l4.x, l4.y))),
                                 y1 = f2_unpack(X ? f2_add(x1, f2_pack(l4.z, l4.w)) : f2_fma(x1, cq2, f2_pack(l4.z, l4.w)));
                    tops[0] = fmaxf(tops[0], y0.x);
                    tops[1] = fmaxf(tops[1], y0.y);
                    tops[2] = fmaxf(tops[2], y1.x);
                    tops[3] = fmaxf(tops[3], y1.y);
                }
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                if (__any_sync(0xffffffffu, top > mref + slack<FMT>())) {
                    const float mn = top > mref + slack<FMT>() ? top - lead<FMT>() : mref, alpha = ex2(mref == -INFINITY ? -INFINITY : mref - mn);
                    mref = mn;
                    mz = mn == -INFINITY ? 0.0f : mn;
                    lsum *= alpha;
                    if (!begins) {            // O of the steps before, once their product is complete
                        gave_up = !__all_sync(0xffffffffu, wait(kPvDone + (b ^ 1), (i - 1) >> 1 & 1));
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16 && !gave_up; ++c) {
                            uint32_t o[16];
                            tc_ld16(tq + kColO + 16 * c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tc_st16(tq + kColO + 16 * c, o);
                        }
                        tc_wait_st();
                    }
                }
                unsigned long long sum0 = f2_pack(lsum, 0.0f), sum1 = zero2;
                const unsigned long long less = f2_pack(-mz, -mz);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pr[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 v4 = *reinterpret_cast<const float4 *>(f + kKeys + 32 * c + j);
                        const int k = 32 * c + j;
                        const unsigned long long x0 = f2_pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1])),
                                                 x1 = f2_pack(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
                        const float2 a0 = f2_unpack(X ? f2_add(x0, less) : f2_fma(x0, cq2, less)),
                                     a1 = f2_unpack(X ? f2_add(x1, less) : f2_fma(x1, cq2, less));
                        const unsigned long long e0 = f2_pack(ex2(a0.x), ex2(a0.y)), e1 = f2_pack(ex2(a1.x), ex2(a1.y));
                        sum0 = f2_add(sum0, e0);
                        sum1 = f2_add(sum1, e1);
                        const float2 p0 = f2_unpack(f2_fma(e0, f2_pack(v4.x, v4.y), zero2)), p1 = f2_unpack(f2_fma(e1, f2_pack(v4.z, v4.w), zero2));
                        pr[j / 2] = pack_h(p0.x, p0.y);
                        pr[j / 2 + 1] = pack_h(p1.x, p1.y);
                    }
                    tc_st16(tq + kColP + 32 * b + 16 * c, pr);
                }
                const float2 sum = f2_unpack(f2_add(sum0, sum1));
                lsum = sum.x + sum.y;
                tc_wait_st();
            }
            if (gave_up) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kPFull + b));
            if (run.f0 + i + 1 < use.end) continue;

            // ---- the segment's end
            if (!__all_sync(0xffffffffu, wait(kPvDone + b, i >> 1 & 1))) break;
            const bool starts = use.base >= run.f0, ends = use.base + use.s.steps <= run.f1, whole = starts && ends;
            if (active) {
                tc_fence_after();
                const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (starts ? 1 : 0)) * A.cols + row;
                const float fo = (FMT == kKv8 ? 0.0625f : 1.0f) * (!whole ? 1.0f : lsum == 0.0f ? 0.0f : 1.0f / lsum);
                const int hq = kvh * A.G + v0 + row - m * A.G;
                __nv_bfloat16 *to = A.out + ((static_cast<size_t>(use.b) * A.M + m) * A.Hq + hq) * D;
                float *po = A.part_o + slot * D;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    tc_ld16(tq + kColO + 16 * c, o);
                    tc_wait_ld();
                    if (row < nv) {
                        float x[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[e]) * fo;
                        if (whole) {
                            uint4 *d = reinterpret_cast<uint4 *>(to + 16 * c);
                            d[0] = make_uint4(pack_b(x[0], x[1]), pack_b(x[2], x[3]), pack_b(x[4], x[5]), pack_b(x[6], x[7]));
                            d[1] = make_uint4(pack_b(x[8], x[9]), pack_b(x[10], x[11]), pack_b(x[12], x[13]), pack_b(x[14], x[15]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                *reinterpret_cast<float4 *>(po + 16 * c + 4 * e) = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                        }
                    }
                }
                if (!whole && row < nv) {
                    A.part_ml[slot * 2] = mref;
                    A.part_ml[slot * 2 + 1] = lsum;
                }
            }
            if (i + 1 == steps) {
                if (threadIdx.x == 0 && !ends && starts)
                    A.info[blockIdx.x] = make_int4(use.b, use.seg, (use.base + use.s.steps - 1) / run.per, 0);
            } else {
                use.next(A, segs);
                fresh = true;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp && keep_tmem == 0) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

template <int FMT, int D, bool X>
cudaError_t launch(const AttnArgs &A, cudaStream_t s, int *grid)
{
    static std::atomic<bool> done[64];          // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev].load()) {
        e = cudaFuncSetAttribute(attn_tc_kernel<FMT, D, X>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<FMT, D>::SMEM);
        if (e != cudaSuccess) return e;
        done[dev].store(true);
    }
    *grid = sm_count();
    attn_tc_kernel<FMT, D, X><<<*grid, kThreads, Tc<FMT, D>::SMEM, s>>>(A);
    return cudaGetLastError();
}
template <int FMT, int D>
cudaError_t launch_x(const AttnArgs &A, cudaStream_t s, int *grid)
{
    return A.softcap > 0.0f || A.slopes ? launch<FMT, D, true>(A, s, grid) : launch<FMT, D, false>(A, s, grid);
}

}  // namespace

cudaError_t attn_tc(int fmt, const AttnArgs &A, cudaStream_t s, int *grid)
{
    if (fmt == kKv4) return A.p.D == 128 ? launch_x<kKv4, 128>(A, s, grid) : launch_x<kKv4, 64>(A, s, grid);
    return A.p.D == 128 ? launch_x<kKv8, 128>(A, s, grid) : launch_x<kKv8, 64>(A, s, grid);
}

}  // namespace nq
