// nq_page_attn_warp.cuh -- the attention kernel whose warps decode for themselves (up
// to 16 query vectors per kv head): see nq_page_attn.cu, which explains and uses it,
// and nq_page_attn_tree.cu (T: trees).
#pragma once

#include <atomic>

#include "nq_page_attn.cuh"

namespace nq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMinRun = 4;              // steps per CTA: one per warp

template <int FMT, int D, int NG, int NT>
struct Geo {
    static constexpr int BASE = block_base(FMT, D, NG), RESID = block_resid(FMT, D);
    // blocks of 16 rows per step.  Two share one maximum and give the MMA four
    // chains: 116 us against 148 with one (4-bit view, 131072 rows of 32 heads)
    static constexpr int BLKS = FMT == kBf16 && D == 128 ? 1 : 2;
    static constexpr int SR = 16 * BLKS;
    static constexpr int STAGE = BLKS * (BASE + RESID);
    // CTAs per SM and stages: as much in flight as shared memory holds beside
    // the merge buffers, three CTAs where registers and two stages fit
    static constexpr int MERGE = D * NT / 4 * 128;                          // accumulators of one warp
    static constexpr int FIX = 2 * MERGE + 2 * 8 * NT * 8;
    static constexpr int fit(int ctas) { return (233472 / ctas - 1024 - 512 - FIX) / (kWarps * STAGE); }
    static constexpr int CTAS = NT == 2 || fit(3) < 2 ? 2 : 3;
    static constexpr int STAGES = fit(CTAS) > 6 ? 6 : fit(CTAS);
    static constexpr int RING = kWarps * STAGES * STAGE;
    static constexpr int SMEM = RING + FIX;
    static_assert(STAGES >= 2, "ring");
};

// X: scores are capped or biased.  T: the last M rows are trees' nodes.
template <int FMT, int D, int NG, int NT, bool X, bool T>
__global__ void __launch_bounds__(kThreads, (Geo<FMT, D, NG, NT>::CTAS))
attn_kernel(const __grid_constant__ AttnArgs A)
{
    using Q = Geo<FMT, D, NG, NT>;
    constexpr int SR = Q::SR, BLKS = Q::BLKS, RB = D / 2, KS = D / 16;
    constexpr int JB = FMT == kBf16 ? 1 : BLKS;                  // blocks per softmax step
    constexpr int NACC = FMT != kBf16 && D == 128 && (NG == 2 || NT == 1) ? 2 : 1;
    constexpr int NGX = FMT == kBf16 ? 1 : NG;
    constexpr int OFF = FMT == kKv8 ? 136 : 8;
    constexpr int TILES = D / 16;
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ __align__(8) unsigned long long bars[kWarps * Q::STAGES];
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int segs = A.p.H * A.QT;
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x < kWarps * Q::STAGES) mbar_init(smem_u32(bars + threadIdx.x), 1);
    if (threadIdx.x == 0) {
        abort_flag = 0;
        A.info[blockIdx.x] = make_int4(-1, 0, 0, 0);             // until the CTA has left a part for the join
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const Run run = find_run<SR, kThreads, D>(A, segs, kMinRun);
    if (run.f0 >= run.f1) return;

    unsigned char *ring = sm + warp * (Q::STAGES * Q::STAGE);
    const uint32_t bar_s = smem_u32(bars + warp * Q::STAGES);
    float *merge = reinterpret_cast<float *>(sm + Q::RING);                      // [2][accumulator][lane]
    float *merge_ml = merge + 2 * Q::MERGE / 4;                                  // [2][column][m, l]
    Walk<SR> use;
    use.open(A, run.b, run.base, run.f0, run.f1);
    int fu = run.f0 + ((warp - (run.f0 & 3)) & 3);               // flat numbers congruent to the warp's
    Feed<FMT, D, NG, BLKS, kWarps> feed;
    feed.start(A, use, segs, fu, smem_u32(ring), bar_s);
    int stage = 0, next_stage = 0, filled = 0;                   // stages that hold or await a step
    uint32_t phase = 0, gone = 0;                                // gone: blocks that are not there, of the filled stages in order
    auto fill = [&]() {
#pragma unroll 1
        for (; filled < Q::STAGES && feed.left > 0; ++filled) {
            feed.issue(A, segs, next_stage, [&](uint32_t out) {
                if (out) gone |= out << (BLKS * filled);
            });
            if (++next_stage == Q::STAGES) next_stage = 0;
        }
    };
    bool fresh = true;                        // a segment (part) begins
    int kvh, v0, nv, all_hi, all_lo, any_hi, any_lo, m_lo, m_hi;
    uint32_t qf[KS][NT][2];
    float cq[NT][2], start[NT][NGX][2], slope2[NT][2], o[TILES][NT][4], mref[NT][2], mz[NT][2], lsum[NT][2];   // mz: mref, 0 for -infinity
    int own[NT][2];                           // row (T: position) of the query itself; rows (own - window, own] are seen
    int mq[T ? NT : 1][2];                    // T: its node
    TreeOf tree;
    const float cap2 = A.softcap * kLog2e, inv2 = X && A.softcap > 0.0f ? 1.0f / cap2 : 0.0f;    // of scores in base 2
    const unsigned window = A.window > 0 ? A.window : 0x7fffffffu;
    for (;;) {
        fill();
        if (fresh) {
        // ================================================= a segment (part)
        fresh = false;
        kvh = use.seg / A.QT;
        v0 = (use.seg - kvh * A.QT) * 8 * NT;
        nv = min(8 * NT, A.M * A.G - v0);
        m_lo = row_of_vector(A, v0);
        m_hi = row_of_vector(A, v0 + nv - 1);
        if constexpr (T) tree = TreeOf(A, use.b, use.s.hi);
        // ---- queries: fragments (column g of each tile), factors and limits of columns 2t, 2t + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int v = v0 + 8 * nt + g;
            const bool valid = v < v0 + nv;
            const int m = valid ? row_of_vector(A, v) : 0, hq = kvh * A.G + (valid ? v - m * A.G : 0);
            const __nv_bfloat16 *qr = A.q + (static_cast<long long>(use.b) * A.M + m) * A.q_stride + hq * D;
            uint32_t fr[KS][2];
            float f = 1.0f;
            if constexpr (FMT == kBf16) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    fr[k][0] = valid ? *reinterpret_cast<const uint32_t *>(qr + 16 * k + 2 * t) : 0u;
                    fr[k][1] = valid ? *reinterpret_cast<const uint32_t *>(qr + 16 * k + 2 * t + 8) : 0u;
                }
            } else {
                // 8 values per word w of the lane's K bytes, in the words' order
                float x[D / 32][8], top = 0.0f;
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    const int d = NG == 2 ? 64 * (w >> 1) + 16 * t + 8 * (w & 1) : (D == 128 ? 32 : 16) * t + 8 * w;
                    const uint4 r = valid ? *reinterpret_cast<const uint4 *>(qr + d) : make_uint4(0, 0, 0, 0);
                    const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[w][2 * j] = __uint_as_float(rw[j] << 16);
                        x[w][2 * j + 1] = __uint_as_float(rw[j] & 0xFFFF0000u);
                        top = fmaxf(top, fmaxf(fabsf(x[w][2 * j]), fabsf(x[w][2 * j + 1])));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int up = min(137 - static_cast<int>(__float_as_uint(top) >> 23), 120);   // largest to [2^10, 2^11)
                const float to = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                f = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
                float sum[NGX] = {};
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[w][j] = __half2float(__float2half_rn(x[w][j] * to));
                        sum[NG == 2 ? w >> 1 : 0] += x[w][j];
                    }
                    constexpr float odd = 1.0f / odd_scale<FMT>();
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        fr[2 * w + s][0] = pack_h(x[w][2 * s], x[w][2 * s + 4]);
                        fr[2 * w + s][1] = pack_h(x[w][2 * s + 1] * odd, x[w][2 * s + 5] * odd);
                    }
                }
#pragma unroll
                for (int gr = 0; gr < NGX; ++gr) {
                    sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
                    sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        start[nt][gr][c] = -static_cast<float>(OFF) * 5.9604644775390625e-08f *
                                           __shfl_sync(0xffffffffu, sum[gr], 4 * (2 * t + c));
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int vc = min(v0 + 8 * nt + 2 * t + c, v0 + nv - 1);
                const float fc = FMT == kBf16 ? 1.0f : __shfl_sync(0xffffffffu, f, 4 * (2 * t + c));
                // undo the codes' 2^-24 (and, for KV8, the 16) and the query's power of two
                cq[nt][c] = A.scale * kLog2e * fc * (FMT == kBf16 ? 1.0f : FMT == kKv8 ? 1048576.0f : 16777216.0f);
                // not 0, which would make NaN of a hidden score: a query of zeros under a tiny scale
                if constexpr (FMT != kBf16) cq[nt][c] = fmaxf(cq[nt][c], 1.2e-38f);
                const int mc = row_of_vector(A, vc);
                own[nt][c] = use.s.hi - A.M + (T ? tree.depth[mc] : mc);
                if constexpr (T) mq[nt][c] = mc;
                slope2[nt][c] = X && A.slopes ? A.slopes[kvh * A.G + vc - mc * A.G] * kLog2e : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][nt][0] = fr[k][0];
                qf[k][nt][1] = fr[k][1];
            }
        }
        // rows that every query of the tile sees: no mask needed there
        all_hi = use.s.hi - A.M + m_lo + 1;
        all_lo = first_seen(A, use.s.hi - A.M + m_hi);
        // rows that any of them sees
        any_hi = use.s.hi - A.M + m_hi + 1;
        any_lo = first_seen(A, use.s.hi - A.M + m_lo);
        if constexpr (T) {                    // depths lie in 0 .. M - 1
            all_hi = tree.base;
            all_lo = first_seen(A, use.s.hi - 1);
            any_hi = use.s.hi;
            any_lo = first_seen(A, tree.base);
        }

#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < TILES; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
            mref[nt][0] = mref[nt][1] = -INFINITY;
            mz[nt][0] = mz[nt][1] = 0.0f;
            lsum[nt][0] = lsum[nt][1] = 0.0f;
        }
        }

        // ================================================= the warp's next step of it
        if (fu < use.end) {
            feed.wait(A, bar_s, stage, phase, Q::STAGES, filled, &abort_flag);
            const int row0 = use.s.lo + (fu - use.base) * SR;
            const unsigned char *sp = ring + stage * Q::STAGE;
            const bool masked = row0 < all_lo || row0 + SR > all_hi || (FMT != kBf16 && (gone & ((1u << BLKS) - 1)) != 0);
#pragma unroll
            for (int j0 = 0; j0 < BLKS; j0 += JB) {
                if (row0 + 16 * j0 >= any_hi) break;             // not copied, or seen by no query
                if (FMT == kBf16 && (gone >> j0 & 1u)) continue;
                // ---- scales of the rows g, g + 8 of each block; log2 of V's
                float sk[JB][2][NGX], sv[JB][2][NGX], lv[JB][2];
                if constexpr (FMT != kBf16) {
#pragma unroll
                    for (int j = 0; j < JB; ++j) {
                        const __half *sc = reinterpret_cast<const __half *>(sp + (j0 + j) * Q::BASE + 32 * RB);
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            const int r = g + 8 * rr;
#pragma unroll
                            for (int gr = 0; gr < NGX; ++gr) {
                                sk[j][rr][gr] = __half2float(sc[r * NG + gr]);
                                sv[j][rr][gr] = __half2float(sc[16 * NG + r * NG + gr]);
                            }
                        }
                    }
                    if (masked) {                                // a row that no query sees may hold anything
#pragma unroll
                        for (int j = 0; j < JB; ++j)
#pragma unroll
                            for (int rr = 0; rr < 2; ++rr) {
                                const bool none = static_cast<unsigned>(row0 + 16 * (j0 + j) + g + 8 * rr - any_lo) >= static_cast<unsigned>(any_hi - any_lo) ||
                                                  (gone >> (j0 + j) & 1u) || (T && !tree.live(row0 + 16 * (j0 + j) + g + 8 * rr));
#pragma unroll
                                for (int gr = 0; gr < NGX; ++gr) {
                                    sk[j][rr][gr] = none ? 0.0f : sk[j][rr][gr];
                                    sv[j][rr][gr] = none ? 0.0f : sv[j][rr][gr];
                                }
                            }
                    }
#pragma unroll
                    for (int j = 0; j < JB; ++j)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr)           // a scale of 0 has codes of 0
                            lv[j][rr] = lg2(fmaxf(NGX == 2 ? fmaxf(sv[j][rr][0], sv[j][rr][NGX - 1]) : sv[j][rr][0], 3.7252902984619140625e-09f));
                }
                // ---- S^T
                float acc[JB][NT][NACC][4];
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    if constexpr (FMT == kBf16) {
                        const unsigned char *bp = sp + (j0 + j) * Q::BASE;
                        const int r = (lane & 7) + 8 * ((lane >> 3) & 1);
                        const uint32_t at = smem_u32(bp) + r * 2 * D;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            uint32_t a0, a1, a2, a3;
                            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                                         : "r"(at + (((2 * k + (lane >> 4)) ^ (r & 7)) << 4)) : "memory");
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (k == 0) mma_from<FMT>(acc[j][nt][0], a0, a1, a2, a3, qf[k][nt][0], qf[k][nt][1], 0.0f, 0.0f);
                                else mma<FMT>(acc[j][nt][0], a0, a1, a2, a3, qf[k][nt][0], qf[k][nt][1]);
                            }
                        }
                    } else {
                        constexpr int NW = D / 32;
                        const unsigned char *bp = sp + (j0 + j) * Q::BASE, *rp = sp + BLKS * Q::BASE + (j0 + j) * Q::RESID;
                        uint32_t kb[2][NW], kr[2][NW];
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            const int r = g + 8 * rr;
                            if constexpr (D == 128 && NG == 1) {
                                const uint4 x = *reinterpret_cast<const uint4 *>(bp + nib_off(RB, r, 16 * t));
                                kb[rr][0] = x.x; kb[rr][1] = x.y; kb[rr][2] = x.z; kb[rr][3] = x.w;
                                if constexpr (FMT == kKv8) {
                                    const uint4 y = *reinterpret_cast<const uint4 *>(rp + nib_off(RB, r, 16 * t));
                                    kr[rr][0] = y.x; kr[rr][1] = y.y; kr[rr][2] = y.z; kr[rr][3] = y.w;
                                }
                            } else {
#pragma unroll
                                for (int h = 0; h < D / 64; ++h) {
                                    const uint2 x = *reinterpret_cast<const uint2 *>(bp + nib_off(RB, r, 32 * h + 8 * t));
                                    kb[rr][2 * h] = x.x; kb[rr][2 * h + 1] = x.y;
                                    if constexpr (FMT == kKv8) {
                                        const uint2 y = *reinterpret_cast<const uint2 *>(rp + nib_off(RB, r, 32 * h + 8 * t));
                                        kr[rr][2 * h] = y.x; kr[rr][2 * h + 1] = y.y;
                                    }
                                }
                            }
                            if constexpr (FMT != kKv8) {
#pragma unroll
                                for (int w = 0; w < NW; ++w) kr[rr][w] = 0u;
                            }
                        }
#pragma unroll
                        for (int w = 0; w < NW; ++w) {
                            const Codes<FMT> c0(kb[0][w], kr[0][w]), c1(kb[1][w], kr[1][w]);
                            constexpr int per_acc = NW / NACC;
                            const int h = w / per_acc;           // the accumulator; its first products start from the offset's
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                const uint32_t a0 = c0.pair(2 * s), a1 = c1.pair(2 * s), a2 = c0.pair(2 * s + 1), a3 = c1.pair(2 * s + 1);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    const uint32_t b0 = qf[2 * w + s][nt][0], b1 = qf[2 * w + s][nt][1];
                                    if (w % per_acc == 0 && s == 0) {
                                        const bool off = NG == 2 || h == 0;
                                        mma_from<FMT>(acc[j][nt][h], a0, a1, a2, a3, b0, b1, off ? start[nt][NG == 2 ? h : 0][0] : 0.0f,
                                                      off ? start[nt][NG == 2 ? h : 0][1] : 0.0f);
                                    } else {
                                        mma<FMT>(acc[j][nt][h], a0, a1, a2, a3, b0, b1);
                                    }
                                }
                            }
                        }
                    }
                }
                // ---- softmax
                uint32_t pb[JB][NT][NGX][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    // scores in base 2 (X), or what cq makes scores of; y: with the log2 of V's scale
                    float s[JB][2][2], y[JB][2][2];
#pragma unroll
                    for (int j = 0; j < JB; ++j)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float x;
                                const int e = 2 * rr + c;
                                if constexpr (FMT == kBf16) x = acc[j][nt][0][e];
                                else if constexpr (NG == 2) x = fmaf(sk[j][rr][1], acc[j][nt][1][e], sk[j][rr][0] * acc[j][nt][0][e]);
                                else x = sk[j][rr][0] * (NACC == 2 ? acc[j][nt][0][e] + acc[j][nt][NACC - 1][e] : acc[j][nt][0][e]);
                                if constexpr (X) {
                                    x *= cq[nt][c];
                                    if (A.softcap > 0.0f) x = capped(x, cap2, inv2);
                                    const int key = row0 + 16 * (j0 + j) + g + 8 * rr;
                                    if (A.slopes) x = fmaf(slope2[nt][c], static_cast<float>((T ? tree.position(key) : key) - own[nt][c]), x);
                                }
                                s[j][rr][c] = x;
                                y[j][rr][c] = FMT == kBf16 ? (X ? x : x * cq[nt][c]) : X ? x + lv[j][rr] : fmaf(x, cq[nt][c], lv[j][rr]);
                            }
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < JB; ++j)
#pragma unroll
                            for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    // before the window, or (negative) after the query's own row
                                    const int key = row0 + 16 * (j0 + j) + g + 8 * rr;
                                    const bool hidden = (T ? !tree.sees(mq[T ? nt : 0][c], own[nt][c], key, window)
                                                           : static_cast<unsigned>(own[nt][c] - key) >= window) ||
                                                        (FMT != kBf16 && (gone >> (j0 + j) & 1u));
                                    s[j][rr][c] = hidden ? -INFINITY : s[j][rr][c];
                                    y[j][rr][c] = hidden ? -INFINITY : y[j][rr][c];
                                }
                    }
                    float top[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        top[c] = fmaxf(y[0][0][c], y[0][1][c]);
#pragma unroll
                        for (int j = 1; j < JB; ++j) top[c] = fmaxf(top[c], fmaxf(y[j][0][c], y[j][1][c]));
                        top[c] = col_max(top[c]);
                    }
                    if (__any_sync(0xffffffffu, top[0] > mref[nt][0] + slack<FMT>() || top[1] > mref[nt][1] + slack<FMT>())) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float mn = top[c] > mref[nt][c] + slack<FMT>() ? top[c] - lead<FMT>() : mref[nt][c];
                            const float alpha = ex2(mref[nt][c] == -INFINITY ? -INFINITY : mref[nt][c] - mn);   // nothing yet: 0
                            mref[nt][c] = mn;
                            mz[nt][c] = mn == -INFINITY ? 0.0f : mn;
                            lsum[nt][c] *= alpha;
#pragma unroll
                            for (int i = 0; i < TILES; ++i) {
                                o[i][nt][c] *= alpha;
                                o[i][nt][2 + c] *= alpha;
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < JB; ++j)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            const float e0 = ex2(X ? s[j][rr][0] - mz[nt][0] : fmaf(s[j][rr][0], cq[nt][0], -mz[nt][0])),
                                        e1 = ex2(X ? s[j][rr][1] - mz[nt][1] : fmaf(s[j][rr][1], cq[nt][1], -mz[nt][1]));
                            if constexpr (FMT == kBf16) {
                                const uint32_t p = pack_b(e0, e1);
                                lsum[nt][0] += __uint_as_float(p << 16);
                                lsum[nt][1] += __uint_as_float(p & 0xFFFF0000u);
                                pb[j][nt][0][rr] = transpose8(p);
                            } else {
                                lsum[nt][0] += e0;
                                lsum[nt][1] += e1;
#pragma unroll
                                for (int gr = 0; gr < NGX; ++gr) pb[j][nt][gr][rr] = transpose8(pack_h(e0 * sv[j][rr][gr], e1 * sv[j][rr][gr]));
                            }
                        }
                }
                // ---- O^T
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    const unsigned char *bp = sp + (j0 + j) * Q::BASE;
                    if constexpr (FMT == kBf16) {
                        const int r = (lane & 7) + 8 * (lane >> 4), blk0 = row0 + 16 * (j0 + j);
                        const uint32_t at = smem_u32(bp) + 32 * D + r * 2 * D;
                        auto product = [&](auto mask_c, uint32_t k0, uint32_t k1, int only) {   // V rows kept; one query row alone, or all
                            constexpr bool MASK = decltype(mask_c)::value;
#pragma unroll
                            for (int i = 0; i < TILES; ++i) {
                                uint32_t a0, a1, a2, a3;
                                asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                                             : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                                             : "r"(at + (((2 * i + ((lane >> 3) & 1)) ^ (r & 7)) << 4)) : "memory");
                                if constexpr (MASK) {
                                    a0 &= k0; a1 &= k0; a2 &= k1; a3 &= k1;
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    if (MASK && only >= 0) {          // 0 times infinity must not reach the other columns
                                        float one[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                        mma<FMT>(one, a0, a1, a2, a3, pb[j][nt][0][0], pb[j][nt][0][1]);
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (row_of_vector(A, v0 + 8 * nt + 2 * t + (e & 1)) == only) o[i][nt][e] += one[e];
                                    } else {
                                        mma<FMT>(o[i][nt], a0, a1, a2, a3, pb[j][nt][0][0], pb[j][nt][0][1]);
                                    }
                                }
                            }
                        };
                        if (masked) {
                            // P is 0 where a query does not see a row, but 0 times NaN or infinity is not:
                            // rows that no query sees (they may hold anything) leave V's fragments.  A
                            // non-finite row that only some queries see is rare; then query row by query row.
                            // rows of [lo, hi); trees: rows that node m sees, or any of them (m < 0)
                            auto kept = [&](int m, int lo, int hi, int k) {
                                const int a = blk0 + 2 * t + 8 * k;
                                if constexpr (T) {
                                    auto keep = [&](int row) {
                                        if (m < 0) return row >= any_lo && row < any_hi && tree.live(row);
                                        return tree.used(m) && tree.sees(m, tree.base + tree.depth[m], row, window);
                                    };
                                    return (keep(a) ? 0x0000FFFFu : 0u) | (keep(a + 1) ? 0xFFFF0000u : 0u);
                                } else {
                                    return (a >= lo && a < hi ? 0x0000FFFFu : 0u) | (a + 1 >= lo && a + 1 < hi ? 0xFFFF0000u : 0u);
                                }
                            };
                            bool bad = false;
                            if (m_hi > m_lo) {
                                const int rr = lane >> 1, key = blk0 + rr;
                                if (key >= any_lo && key < any_hi && !(key >= all_lo && key < all_hi) && (!T || tree.live(key))) {
                                    const uint4 *x = reinterpret_cast<const uint4 *>(bp + 32 * D + rr * 2 * D) + (lane & 1) * (D / 16);
#pragma unroll 4
                                    for (int i = 0; i < D / 16; ++i) {
                                        const uint4 y = x[i];
                                        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                                        for (int u = 0; u < 4; ++u)
                                            bad |= (w[u] & 0x7F80u) == 0x7F80u || (w[u] & 0x7F800000u) == 0x7F800000u;
                                    }
                                }
                            }
                            if (__any_sync(0xffffffffu, bad)) {
                                for (int m = m_lo; m <= m_hi; ++m) {
                                    const int hi = use.s.hi - A.M + m + 1, lo = first_seen(A, hi - 1);   // without trees: of query m
                                    product(std::true_type{}, kept(m, lo, hi, 0), kept(m, lo, hi, 1), m);
                                }
                            } else {
                                product(std::true_type{}, kept(-1, any_lo, any_hi, 0), kept(-1, any_lo, any_hi, 1), -1);
                            }
                        } else {
                            product(std::false_type{}, 0u, 0u, -1);
                        }
                    } else {
                        constexpr int NW = D / 64;
                        const unsigned char *rp = sp + BLKS * Q::BASE + (j0 + j) * Q::RESID;
                        uint32_t vb[4][NW], vr[4][NW];
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const int r = 2 * t + (kk & 1) + 8 * (kk >> 1);
                            if constexpr (D == 128 && NG == 1) {
                                const uint2 x = *reinterpret_cast<const uint2 *>(bp + 16 * RB + nib_off(RB, r, 8 * g));
                                vb[kk][0] = x.x; vb[kk][1] = x.y;
                                if constexpr (FMT == kKv8) {
                                    const uint2 y = *reinterpret_cast<const uint2 *>(rp + 16 * RB + nib_off(RB, r, 8 * g));
                                    vr[kk][0] = y.x; vr[kk][1] = y.y;
                                }
                            } else {
#pragma unroll
                                for (int h = 0; h < NW; ++h) {
                                    vb[kk][h] = *reinterpret_cast<const uint32_t *>(bp + 16 * RB + nib_off(RB, r, 32 * h + 4 * g));
                                    if constexpr (FMT == kKv8)
                                        vr[kk][h] = *reinterpret_cast<const uint32_t *>(rp + 16 * RB + nib_off(RB, r, 32 * h + 4 * g));
                                }
                            }
                            if constexpr (FMT != kKv8) {
#pragma unroll
                                for (int h = 0; h < NW; ++h) vr[kk][h] = 0u;
                            }
                        }
#pragma unroll
                        for (int w = 0; w < NW; ++w) {
                            // nibbles of rows 2t | 2t + 1 and 2t + 8 | 2t + 9 side by side
                            const Codes<FMT> x0(__byte_perm(vb[0][w], vb[1][w], 0x5410), __byte_perm(vr[0][w], vr[1][w], 0x5410)),
                                x1(__byte_perm(vb[0][w], vb[1][w], 0x7632), __byte_perm(vr[0][w], vr[1][w], 0x7632)),
                                y0(__byte_perm(vb[2][w], vb[3][w], 0x5410), __byte_perm(vr[2][w], vr[3][w], 0x5410)),
                                y1(__byte_perm(vb[2][w], vb[3][w], 0x7632), __byte_perm(vr[2][w], vr[3][w], 0x7632));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t a0 = x0.value(i), a1 = x1.value(i), a2 = y0.value(i), a3 = y1.value(i);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma<FMT>(o[4 * w + i][nt], a0, a1, a2, a3, pb[j][nt][NG == 2 ? w : 0][0], pb[j][nt][NG == 2 ? w : 0][1]);
                            }
                        }
                    }
                }
            }
            // the stage was read through the generic proxy, the next copy writes through the async one
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            --filled;
            gone >>= BLKS;
            fu += kWarps;
            if (++stage == Q::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            if (fu < use.end) continue;
        }

        // ================================================= the segment's end: the warps merge
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            lsum[nt][0] = col_sum(lsum[nt][0]);
            lsum[nt][1] = col_sum(lsum[nt][1]);
        }
        auto put = [&](int buf) {
            float *d = merge + buf * (Q::MERGE / 4) + lane;
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[((i * NT + nt) * 4 + e) * 32] = o[i][nt][e];
            if (g == 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        merge_ml[(buf * 8 * NT + 8 * nt + 2 * t + c) * 2] = mref[nt][c];
                        merge_ml[(buf * 8 * NT + 8 * nt + 2 * t + c) * 2 + 1] = lsum[nt][c];
                    }
            }
        };
        auto take = [&](int buf) {
            const float *d = merge + buf * (Q::MERGE / 4) + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float fa[2], fb[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float mb = merge_ml[(buf * 8 * NT + 8 * nt + 2 * t + c) * 2], lb = merge_ml[(buf * 8 * NT + 8 * nt + 2 * t + c) * 2 + 1];
                    const float mn = fmaxf(mref[nt][c], mb), mz = mn == -INFINITY ? 0.0f : mn;
                    fa[c] = ex2(mref[nt][c] - mz);
                    fb[c] = ex2(mb - mz);
                    mref[nt][c] = mn;
                    lsum[nt][c] = lsum[nt][c] * fa[c] + lb * fb[c];
                }
#pragma unroll
                for (int i = 0; i < TILES; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[i][nt][e] = o[i][nt][e] * fa[e & 1] + d[((i * NT + nt) * 4 + e) * 32] * fb[e & 1];
            }
        };
        // warps 2, 3 to 0, 1, then 1 to 0; the first barrier also frees the buffers of the segment before
#pragma unroll 1
        for (int half = 2; half > 0; half >>= 1) {
            __syncthreads();
            if (warp >= half && warp < 2 * half) put(warp - half);
            __syncthreads();
            if (warp < half) take(warp);
        }
        if (warp == 0) {
            const bool starts = use.base >= run.f0, ends = use.base + use.s.steps <= run.f1, whole = starts && ends;
            if (!ends && starts && lane == 0 && *const_cast<volatile int *>(&abort_flag) == 0)
                A.info[blockIdx.x] = make_int4(use.b, use.seg, (use.base + use.s.steps - 1) / run.per, 0);
            const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (starts ? 1 : 0);
            constexpr float unit = FMT == kKv8 ? 0.0625f : 1.0f;                 // KV8's codes are 16 times the value
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = 8 * nt + 2 * t + c;
                    if (col >= nv) continue;
                    if constexpr (T)
                        if (!tree.used(mq[nt][c])) {             // its query may have been anything
                            mref[nt][c] = -INFINITY;
                            lsum[nt][c] = 0.0f;
#pragma unroll
                            for (int i = 0; i < TILES; ++i) o[i][nt][c] = o[i][nt][2 + c] = 0.0f;
                        }
                    const float f = unit * (!whole ? 1.0f : lsum[nt][c] == 0.0f ? 0.0f : 1.0f / lsum[nt][c]);
                    const int v = v0 + col, m = row_of_vector(A, v);
                    __nv_bfloat16 *to = A.out + ((static_cast<size_t>(use.b) * A.M + m) * A.Hq + kvh * A.G + v - m * A.G) * D;
                    float *po = A.part_o + (slot * 8 * NT + col) * D;
                    if (!whole && g == 0) {
                        A.part_ml[(slot * 8 * NT + col) * 2] = mref[nt][c];
                        A.part_ml[(slot * 8 * NT + col) * 2 + 1] = lsum[nt][c];
                    }
                    if constexpr (FMT == kBf16) {
#pragma unroll
                        for (int i = 0; i < TILES; ++i)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                if (whole) to[16 * i + 8 * r + g] = __float2bfloat16_rn(o[i][nt][2 * r + c] * f);
                                else po[16 * i + 8 * r + g] = o[i][nt][2 * r + c] * f;
                            }
                    } else {
                        // a lane's eight values of word w: dimensions d .. d + 7
#pragma unroll
                        for (int w = 0; w < D / 64; ++w) {
                            const int d = D == 128 && NG == 1 ? 16 * g + 8 * w : 64 * w + 8 * g;
                            float x[8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                x[i] = o[4 * w + i][nt][c] * f;
                                x[4 + i] = o[4 * w + i][nt][2 + c] * f;
                            }
                            if (whole) {
                                *reinterpret_cast<uint4 *>(to + d) = make_uint4(pack_b(x[0], x[1]), pack_b(x[2], x[3]),
                                                                                pack_b(x[4], x[5]), pack_b(x[6], x[7]));
                            } else {
                                *reinterpret_cast<float4 *>(po + d) = make_float4(x[0], x[1], x[2], x[3]);
                                *reinterpret_cast<float4 *>(po + d + 4) = make_float4(x[4], x[5], x[6], x[7]);
                            }
                        }
                    }
                }
        }
        if (use.end >= use.stop) break;
        use.next(A, segs);
        fresh = true;
    }
}

template <int FMT, int D, int NG, int NT, bool X, bool T>
cudaError_t launch(const AttnArgs &A, cudaStream_t s, int *grid)
{
    using Q = Geo<FMT, D, NG, NT>;
    static std::atomic<bool> done[64];          // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev].load()) {
        e = cudaFuncSetAttribute(attn_kernel<FMT, D, NG, NT, X, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q::SMEM);
        if (e != cudaSuccess) return e;
        done[dev].store(true);
    }
    *grid = sm_count() * Q::CTAS;
    attn_kernel<FMT, D, NG, NT, X, T><<<*grid, kThreads, Q::SMEM, s>>>(A);
    return cudaGetLastError();
}
// (Trees take the form for capped or biased scores whatever theirs are.)
template <int FMT, int D, int NG, bool T>
cudaError_t launch_x(int nt, const AttnArgs &A, cudaStream_t s, int *grid)
{
    if (T || A.softcap > 0.0f || A.slopes) return nt == 1 ? launch<FMT, D, NG, 1, true, T>(A, s, grid) : launch<FMT, D, NG, 2, true, T>(A, s, grid);
    if constexpr (!T) return nt == 1 ? launch<FMT, D, NG, 1, false, T>(A, s, grid) : launch<FMT, D, NG, 2, false, T>(A, s, grid);
}
template <int FMT, bool T>
cudaError_t launch_d(int nt, const AttnArgs &A, cudaStream_t s, int *grid)
{
    if (A.p.D == 64) return launch_x<FMT, 64, 1, T>(nt, A, s, grid);
    if constexpr (FMT != kBf16)
        if (A.p.NG == 2) return launch_x<FMT, 128, 2, T>(nt, A, s, grid);
    return launch_x<FMT, 128, 1, T>(nt, A, s, grid);
}

}  // namespace
}  // namespace nq
