// nq_page_attn_wide.cuh -- the attention kernel whose CTAs decode a step once for
// all their query vectors: see nq_page_attn_wide.cu, which explains and uses it, and
// nq_page_attn_tree_wide.cu (T: trees).
#pragma once

#include <atomic>

#include "nq_page_attn.cuh"

namespace nq {
namespace {

constexpr int kMinRun = 2;              // steps per CTA

template <int FMT, int D, int NG, int WARPS>
struct Wide {
    static constexpr int BASE = block_base(FMT, D, NG), RESID = block_resid(FMT, D);
    static constexpr int BLKS = 2, SR = 32;
    static constexpr int STAGE = BLKS * (BASE + RESID);
    static constexpr int TILE = 16 * D * 2;                                  // 16 rows of K (or V) in 16 bits
    static constexpr int SCALES = FMT == kBf16 ? 0 : BLKS * 64 * NG;         // of a step, as in the blocks
    static constexpr int DECODED = FMT == kBf16 ? 0 : 2 * BLKS * TILE + (SCALES + 255) / 256 * 256;   // tiles at multiples of 256
    static constexpr int CTAS = 16 / WARPS;                                  // 16 warps of 128 registers per SM
    static constexpr int FIT = (233472 / CTAS - 1024 - 512 - 2 * DECODED) / STAGE;
    static constexpr int STAGES = FIT > 6 ? 6 : FIT;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int SMEM = RING + 2 * DECODED;
    static_assert(STAGES >= 2, "ring");
};

__device__ __forceinline__ void ldsm(uint32_t at, uint32_t &a0, uint32_t &a1, uint32_t &a2, uint32_t &a3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t at, uint32_t &a0, uint32_t &a1, uint32_t &a2, uint32_t &a3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3) : "r"(at) : "memory");
}
// A decoded row holds the eight values of a word as nibbles 0 4 1 5 2 6 3 7, the
// order in which masks give them: dimension of position p.
template <int FMT>
__device__ __forceinline__ int dim_at(int p)
{
    return FMT == kBf16 ? p : (p & ~7) + ((p & 7) >> 1) + 4 * (p & 1);
}

// X: scores are capped or biased.  T: the last M rows are trees' nodes.
template <int FMT, int D, int NG, int WARPS, bool X, bool T>
__global__ void __launch_bounds__(WARPS * 32, (Wide<FMT, D, NG, WARPS>::CTAS))
attn_wide_kernel(const __grid_constant__ AttnArgs A)
{
    using Q = Wide<FMT, D, NG, WARPS>;
    constexpr int SR = Q::SR, BLKS = Q::BLKS, KS = D / 16, TILES = D / 16, NGX = FMT == kBf16 ? 1 : NG, COLS = 8 * WARPS, THREADS = 32 * WARPS;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ __align__(8) unsigned long long bars[Q::STAGES];
    __shared__ uint32_t gone_of[Q::STAGES], gone_decoded[2];                 // blocks that are not there
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int segs = A.p.H * A.QT;
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x < Q::STAGES) mbar_init(smem_u32(bars + threadIdx.x), 1);
    if (threadIdx.x == 0) {
        abort_flag = 0;
        A.info[blockIdx.x] = make_int4(-1, 0, 0, 0);             // until the CTA has left a part for the join
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const Run run = find_run<SR, THREADS, D>(A, segs, kMinRun);
    if (run.f0 >= run.f1) return;
    unsigned char *decoded = sm, *ring = sm + 2 * Q::DECODED;
    const uint32_t ring_s = smem_u32(ring), bar_s = smem_u32(bars);
    Walk<SR> use;
    use.open(A, run.b, run.base, run.f0, run.f1);
    Feed<FMT, D, NG, BLKS, 1> feed;           // of warp 0
    feed.left = 0;
    int filled = 0, next_stage = 0;
    if (warp == 0) feed.start(A, use, segs, run.f0, ring_s, bar_s);
    auto fill = [&]() {
#pragma unroll 1
        for (; filled < Q::STAGES && feed.left > 0; ++filled) {
            feed.issue(A, segs, next_stage, [&](uint32_t out) { gone_of[next_stage] = out; });
            if (++next_stage == Q::STAGES) next_stage = 0;
        }
    };
    if (warp == 0) fill();

    // step number f of the run into buffer f % 2: thread = (row, quarter of the row) of K, then of V
    int stage = 0;                            // of the next step to be waited for
    uint32_t phase = 0;
    auto wait = [&]() { feed.wait(A, bar_s, stage, phase, Q::STAGES, filled, &abort_flag); };
    auto advance = [&]() {
        if (++stage == Q::STAGES) {
            stage = 0;
            phase ^= 1u;
        }
    };
    auto decode = [&](int buf) {
        if constexpr (FMT != kBf16) {
            constexpr int RB = D / 2, CH = RB / 16;                          // 16-byte chunks of a row of nibbles
            const unsigned char *sp = ring + stage * Q::STAGE;
            unsigned char *out = decoded + buf * Q::DECODED;
#pragma unroll 1
            for (int i = threadIdx.x; i < 2 * SR * CH; i += THREADS) {
                const int v = i / (SR * CH), r = i / CH % SR, c = i % CH, at = (r >> 4) * Q::BASE + v * 16 * RB + nib_off(RB, r & 15, 16 * c);
                const uint4 b = *reinterpret_cast<const uint4 *>(sp + at);
                uint4 x = make_uint4(0, 0, 0, 0);
                if constexpr (FMT == kKv8)
                    x = *reinterpret_cast<const uint4 *>(sp + BLKS * Q::BASE + (r >> 4) * Q::RESID + v * 16 * RB + nib_off(RB, r & 15, 16 * c));
                const uint32_t bw[4] = {b.x, b.y, b.z, b.w}, xw[4] = {x.x, x.y, x.z, x.w};
                unsigned char *to = out + (v * BLKS + (r >> 4)) * Q::TILE + (r & 15) * 2 * D;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const Codes<FMT> k(bw[w], xw[w]);
                    *reinterpret_cast<uint4 *>(to + (((4 * c + w) ^ (r & 7)) << 4)) = make_uint4(k.value(0), k.value(1), k.value(2), k.value(3));
                }
            }
            if (threadIdx.x == 0) gone_decoded[buf] = gone_of[stage];
            constexpr int SC = BLKS * 64 * NG / 16;                          // the scales' 16-byte chunks
            if (threadIdx.x < SC) {
                const int j = threadIdx.x / (4 * NG), k = threadIdx.x % (4 * NG);
                *reinterpret_cast<uint4 *>(out + 2 * BLKS * Q::TILE + threadIdx.x * 16) = *reinterpret_cast<const uint4 *>(sp + j * Q::BASE + 32 * RB + 16 * k);
            }
        }
    };

    bool fresh = true;
    int kvh, v0, nv, all_hi, all_lo, any_hi, any_lo, m_lo, m_hi;
    bool mine = false;
    uint32_t qf[KS][2];
    float cq[2], slope2[2], o[TILES][4], mref[2], mz[2], lsum[2];            // mz: mref, 0 for -infinity
    int own[2];                               // row (T: position) of the query itself
    int mq[2];                                // T: its node
    TreeOf tree;
    const float cap2 = A.softcap * kLog2e, inv2 = X && A.softcap > 0.0f ? 1.0f / cap2 : 0.0f;
    const unsigned window = A.window > 0 ? A.window : 0x7fffffffu;

    if constexpr (FMT != kBf16) {
        wait();
        decode(0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        advance();
        __syncthreads();
        if (warp == 0) {
            --filled;
            fill();
        }
    }
    for (int f = run.f0; f < run.f1; ++f) {
        if (fresh) {
            // ============================================= a segment (part): this warp's columns
            fresh = false;
            kvh = use.seg / A.QT;
            v0 = (use.seg - kvh * A.QT) * COLS;
            nv = min(COLS, A.M * A.G - v0);
            if constexpr (T) tree = TreeOf(A, use.b, use.s.hi);
            mine = 8 * warp < nv;             // columns 8 warp .. 8 warp + 7 of the tile are the warp's
            m_lo = row_of_vector(A, v0);
            m_hi = row_of_vector(A, v0 + nv - 1);
            const int c0 = 8 * warp;
            const bool valid = c0 + g < nv;
            const int v = v0 + c0 + g, m = valid ? row_of_vector(A, v) : 0, hq = kvh * A.G + (valid ? v - m * A.G : 0);
            const __nv_bfloat16 *qr = A.q + (static_cast<long long>(use.b) * A.M + m) * A.q_stride + hq * D;
            float f2 = 1.0f;
            if constexpr (FMT == kBf16) {
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        qf[k][h] = valid ? *reinterpret_cast<const uint32_t *>(qr + 16 * k + 2 * t + 8 * h) : 0u;
            } else {
                float x[KS][2][2], top = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            x[k][h][e] = valid ? __bfloat162float(qr[16 * k + 8 * h + t + 4 * e]) : 0.0f;   // dim_at(2 t + e)
                            top = fmaxf(top, fabsf(x[k][h][e]));
                        }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // largest magnitude to [2^10, 2^11) by a power of two, undone per column
                const int up = min(137 - static_cast<int>(__float_as_uint(top) >> 23), 120);
                const float to = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                f2 = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int h = 0; h < 2; ++h) qf[k][h] = pack_h(x[k][h][0] * to, x[k][h][1] * to);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                cq[c] = A.scale * kLog2e * (FMT == kKv8 ? 0.0625f : 1.0f);
                if constexpr (FMT != kBf16) cq[c] = fmaxf(cq[c] * __shfl_sync(0xffffffffu, f2, 4 * (2 * t + c)), 1.2e-38f);
                const int vc = min(v0 + c0 + 2 * t + c, v0 + nv - 1), mc = row_of_vector(A, vc);
                own[c] = use.s.hi - A.M + (T ? tree.depth[mc] : mc);
                if constexpr (T) mq[c] = mc;
                slope2[c] = X && A.slopes ? A.slopes[kvh * A.G + vc - mc * A.G] * kLog2e : 0.0f;
                mref[c] = -INFINITY;
                mz[c] = 0.0f;
                lsum[c] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < TILES; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
            all_hi = use.s.hi - A.M + m_lo + 1;
            all_lo = first_seen(A, use.s.hi - A.M + m_hi);
            any_hi = use.s.hi - A.M + m_hi + 1;
            any_lo = first_seen(A, use.s.hi - A.M + m_lo);
            if constexpr (T) {                // depths lie in 0 .. M - 1
                all_hi = tree.base;
                all_lo = first_seen(A, use.s.hi - 1);
                any_hi = use.s.hi;
                any_lo = first_seen(A, tree.base);
            }
        }
        const int buf = (f - run.f0) & 1;
        const unsigned char *ktile, *vtile;
        int tile_step;
        uint32_t gone;
        const __half *scales = nullptr;
        if constexpr (FMT == kBf16) {
            wait();
            gone = gone_of[stage];
            ktile = ring + stage * Q::STAGE;
            vtile = ktile + Q::TILE;
            tile_step = Q::BASE;
        } else {
            if (f + 1 < run.f1) {
                wait();
                decode(buf ^ 1);
                advance();
            }
            gone = gone_decoded[buf];
            ktile = decoded + buf * Q::DECODED;
            vtile = ktile + BLKS * Q::TILE;
            tile_step = Q::TILE;
            scales = reinterpret_cast<const __half *>(ktile + 2 * BLKS * Q::TILE);
        }
        const int row0 = use.s.lo + (f - use.base) * SR;
        if (mine && row0 < any_hi) {
            // ---- S^T of both blocks, per group of K's scales
            float acc[BLKS][NGX][4];
            {
                // chunk 2 k + lane / 16 of row r lies at that xor r % 8; rows are aligned, so k enters by an xor
                const int r = (lane & 7) + 8 * ((lane >> 3) & 1);
                const uint32_t at = smem_u32(ktile) + r * 2 * D + (((lane >> 4) ^ (r & 7)) << 4);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int j = 0; j < BLKS; ++j) {
                        uint32_t a0, a1, a2, a3;
                        ldsm((at ^ (32 * k)) + j * tile_step, a0, a1, a2, a3);
                        constexpr int per = KS / NGX;
                        if (k % per == 0) mma_from<FMT>(acc[j][k / per], a0, a1, a2, a3, qf[k][0], qf[k][1], 0.0f, 0.0f);
                        else mma<FMT>(acc[j][k / per], a0, a1, a2, a3, qf[k][0], qf[k][1]);
                    }
            }
            const bool masked = row0 < all_lo || row0 + SR > all_hi || gone != 0;
            float sk[BLKS][2][NGX], sv[BLKS][2][NGX], lv[BLKS][2];
            if constexpr (FMT != kBf16) {
#pragma unroll
                for (int j = 0; j < BLKS; ++j)
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                        for (int gr = 0; gr < NGX; ++gr) {
                            sk[j][rr][gr] = __half2float(scales[32 * NG * j + (g + 8 * rr) * NG + gr]);
                            sv[j][rr][gr] = __half2float(scales[32 * NG * j + 16 * NG + (g + 8 * rr) * NG + gr]);
                        }
                if (masked) {                                    // a row that no query sees may hold anything
#pragma unroll
                    for (int j = 0; j < BLKS; ++j)
#pragma unroll
                        for (int rr = 0; rr < 2; ++rr) {
                            const bool none = static_cast<unsigned>(row0 + 16 * j + g + 8 * rr - any_lo) >= static_cast<unsigned>(any_hi - any_lo) || (gone >> j & 1u) ||
                                              (T && !tree.live(row0 + 16 * j + g + 8 * rr));
#pragma unroll
                            for (int gr = 0; gr < NGX; ++gr) {
                                sk[j][rr][gr] = none ? 0.0f : sk[j][rr][gr];
                                sv[j][rr][gr] = none ? 0.0f : sv[j][rr][gr];
                            }
                        }
                }
#pragma unroll
                for (int j = 0; j < BLKS; ++j)
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr)
                        lv[j][rr] = lg2(fmaxf(NGX == 2 ? fmaxf(sv[j][rr][0], sv[j][rr][NGX - 1]) : sv[j][rr][0], 3.7252902984619140625e-09f));
            }
            // ---- softmax: scores in base 2 (X), or what cq makes scores of; y: with the log2 of V's scale
            float s[BLKS][2][2], y[BLKS][2][2];
#pragma unroll
            for (int j = 0; j < BLKS; ++j)
#pragma unroll
                for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int e = 2 * rr + c;
                        float x;
                        if constexpr (FMT == kBf16) x = acc[j][0][e];
                        else if constexpr (NG == 2) x = fmaf(sk[j][rr][1], acc[j][1][e], sk[j][rr][0] * acc[j][0][e]);
                        else x = sk[j][rr][0] * acc[j][0][e];
                        if constexpr (X) {
                            x *= cq[c];
                            if (A.softcap > 0.0f) x = capped(x, cap2, inv2);
                            const int key = row0 + 16 * j + g + 8 * rr;
                            if (A.slopes) x = fmaf(slope2[c], static_cast<float>((T ? tree.position(key) : key) - own[c]), x);
                        }
                        s[j][rr][c] = x;
                        y[j][rr][c] = FMT == kBf16 ? (X ? x : x * cq[c]) : X ? x + lv[j][rr] : fmaf(x, cq[c], lv[j][rr]);
                    }
            if (masked) {
#pragma unroll
                for (int j = 0; j < BLKS; ++j)
#pragma unroll
                    for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            // before the window, or (negative) after the query's own row
                            const int key = row0 + 16 * j + g + 8 * rr;
                            const bool hidden = (T ? !tree.sees(mq[c], own[c], key, window) : static_cast<unsigned>(own[c] - key) >= window) || (gone >> j & 1u);
                            s[j][rr][c] = hidden ? -INFINITY : s[j][rr][c];
                            y[j][rr][c] = hidden ? -INFINITY : y[j][rr][c];
                        }
            }
            float top[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) top[c] = col_max(fmaxf(fmaxf(y[0][0][c], y[0][1][c]), fmaxf(y[1][0][c], y[1][1][c])));
            if (__any_sync(0xffffffffu, top[0] > mref[0] + slack<FMT>() || top[1] > mref[1] + slack<FMT>())) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float mn = top[c] > mref[c] + slack<FMT>() ? top[c] - lead<FMT>() : mref[c];
                    const float alpha = ex2(mref[c] == -INFINITY ? -INFINITY : mref[c] - mn);    // nothing yet: 0
                    mref[c] = mn;
                    mz[c] = mn == -INFINITY ? 0.0f : mn;
                    lsum[c] *= alpha;
#pragma unroll
                    for (int i = 0; i < TILES; ++i) {
                        o[i][c] *= alpha;
                        o[i][2 + c] *= alpha;
                    }
                }
            }
            uint32_t pb[BLKS][NGX][2];
#pragma unroll
            for (int j = 0; j < BLKS; ++j)
#pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
                    const float e0 = ex2(X ? s[j][rr][0] - mz[0] : fmaf(s[j][rr][0], cq[0], -mz[0])),
                                e1 = ex2(X ? s[j][rr][1] - mz[1] : fmaf(s[j][rr][1], cq[1], -mz[1]));
                    if constexpr (FMT == kBf16) {
                        const uint32_t p = pack_b(e0, e1);
                        lsum[0] += __uint_as_float(p << 16);
                        lsum[1] += __uint_as_float(p & 0xFFFF0000u);
                        pb[j][0][rr] = transpose8(p);
                    } else {
                        lsum[0] += e0;
                        lsum[1] += e1;
#pragma unroll
                        for (int gr = 0; gr < NGX; ++gr) pb[j][gr][rr] = transpose8(pack_h(e0 * sv[j][rr][gr], e1 * sv[j][rr][gr]));
                    }
                }
            // ---- O^T
            const int r = (lane & 7) + 8 * (lane >> 4);
            const uint32_t vrow = smem_u32(vtile) + r * 2 * D + ((((lane >> 3) & 1) ^ (r & 7)) << 4);
            if (FMT == kBf16 && masked) {
                // rows that no query sees (they may hold anything) leave V; a non-finite row that
                // only some queries see is rare: then query row by query row (0 times infinity)
#pragma unroll 1
                for (int j = 0; j < BLKS; ++j) {
                    if (gone >> j & 1u) continue;
                    const int blk0 = row0 + 16 * j;
                    // rows of [lo, hi); trees: of the rows that node m sees, those of [lo, hi) for m < 0.  (Bounds that the
                    // caller forms: formed in here, heads of 128 under a cap spill more, 71.5 us against 66.5 for 20 vectors.)
                    auto kept = [&](int m, int lo, int hi, int k) {
                        const int a = blk0 + 2 * t + 8 * k;
                        if constexpr (T) {
                            auto keep = [&](int row) {
                                if (m >= 0) return tree.used(m) && tree.sees(m, tree.base + tree.depth[m], row, window);
                                return row >= lo && row < hi && tree.live(row);
                            };
                            return (keep(a) ? 0x0000FFFFu : 0u) | (keep(a + 1) ? 0xFFFF0000u : 0u);
                        } else {
                            return (a >= lo && a < hi ? 0x0000FFFFu : 0u) | (a + 1 >= lo && a + 1 < hi ? 0xFFFF0000u : 0u);
                        }
                    };
                    bool bad = false;
                    const int rr = lane >> 1, key = blk0 + rr;
                    if (key >= any_lo && key < any_hi && !(key >= all_lo && key < all_hi) && (!T || tree.live(key))) {
                        const uint4 *x = reinterpret_cast<const uint4 *>(vtile + j * tile_step + rr * 2 * D) + (lane & 1) * (D / 16);
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) {
                            const uint4 w = x[i];
                            bad |= (w.x & 0x7F80u) == 0x7F80u || (w.x & 0x7F800000u) == 0x7F800000u || (w.y & 0x7F80u) == 0x7F80u ||
                                   (w.y & 0x7F800000u) == 0x7F800000u || (w.z & 0x7F80u) == 0x7F80u || (w.z & 0x7F800000u) == 0x7F800000u ||
                                   (w.w & 0x7F80u) == 0x7F80u || (w.w & 0x7F800000u) == 0x7F800000u;
                        }
                    }
                    bad = __any_sync(0xffffffffu, bad);
                    const uint32_t p0 = j ? pb[BLKS - 1][0][0] : pb[0][0][0], p1 = j ? pb[BLKS - 1][0][1] : pb[0][0][1];
#pragma unroll 1
                    for (int m = bad ? m_lo : m_hi; m <= m_hi; ++m) {
                        const int at = use.s.hi - A.M + m;       // without trees: the row of query m
                        const uint32_t k0 = bad ? kept(m, first_seen(A, at), at + 1, 0) : kept(-1, any_lo, any_hi, 0);
                        const uint32_t k1 = bad ? kept(m, first_seen(A, at), at + 1, 1) : kept(-1, any_lo, any_hi, 1);
#pragma unroll
                        for (int i = 0; i < TILES; ++i) {
                            uint32_t a0, a1, a2, a3;
                            ldsm_t((vrow ^ (32 * i)) + j * tile_step, a0, a1, a2, a3);
                            float one[4];
                            mma_from<FMT>(one, a0 & k0, a1 & k0, a2 & k1, a3 & k1, p0, p1, 0.0f, 0.0f);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!bad || row_of_vector(A, v0 + 8 * warp + 2 * t + (e & 1)) == m) o[i][e] += one[e];
                        }
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < BLKS; ++j)
#pragma unroll
                    for (int i = 0; i < TILES; ++i) {
                        uint32_t a0, a1, a2, a3;
                        ldsm_t((vrow ^ (32 * i)) + j * tile_step, a0, a1, a2, a3);
                        mma<FMT>(o[i], a0, a1, a2, a3, pb[j][i * NGX / TILES][0], pb[j][i * NGX / TILES][1]);
                    }
            }
        }
        // read through the generic proxy here, written through the async one by the copy that follows
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        if constexpr (FMT == kBf16) advance();
        if (warp == 0) {
            --filled;
            fill();
        }
        if (f + 1 < use.end) continue;

        // ================================================= the segment's end
        const bool starts = use.base >= run.f0, ends = use.base + use.s.steps <= run.f1, whole = starts && ends;
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (starts ? 1 : 0);
        constexpr float unit = FMT == kKv8 ? 0.0625f : 1.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            lsum[c] = col_sum(lsum[c]);
            const int col = 8 * warp + 2 * t + c;
            if (col >= nv) continue;
            if constexpr (T)
                if (!tree.used(mq[c])) {      // its query may have been anything
                    mref[c] = -INFINITY;
                    lsum[c] = 0.0f;
#pragma unroll
                    for (int i = 0; i < TILES; ++i) o[i][c] = o[i][2 + c] = 0.0f;
                }
            const float fo = unit * (!whole ? 1.0f : lsum[c] == 0.0f ? 0.0f : 1.0f / lsum[c]);
            const int v = v0 + col, m = row_of_vector(A, v);
            __nv_bfloat16 *to = A.out + ((static_cast<size_t>(use.b) * A.M + m) * A.Hq + kvh * A.G + v - m * A.G) * D;
            float *po = A.part_o + (slot * COLS + col) * D;
            if (!whole && g == 0) {
                A.part_ml[(slot * COLS + col) * 2] = mref[c];
                A.part_ml[(slot * COLS + col) * 2 + 1] = lsum[c];
            }
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int d = 16 * i + 8 * r + dim_at<FMT>(g);
                    if (whole) to[d] = __float2bfloat16_rn(o[i][2 * r + c] * fo);
                    else po[d] = o[i][2 * r + c] * fo;
                }
        }
        if (f + 1 == run.f1) {
            if (threadIdx.x == 0 && !ends && starts && *const_cast<volatile int *>(&abort_flag) == 0)
                A.info[blockIdx.x] = make_int4(use.b, use.seg, (use.base + use.s.steps - 1) / run.per, 0);
        } else {
            use.next(A, segs);
            fresh = true;
        }
    }
}

template <int FMT, int D, int NG, int WARPS, bool X, bool T>
cudaError_t launch(const AttnArgs &A, cudaStream_t s, int *grid)
{
    using Q = Wide<FMT, D, NG, WARPS>;
    static std::atomic<bool> done[64];          // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev].load()) {
        e = cudaFuncSetAttribute(attn_wide_kernel<FMT, D, NG, WARPS, X, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q::SMEM);
        if (e != cudaSuccess) return e;
        done[dev].store(true);
    }
    *grid = sm_count() * Q::CTAS;
    attn_wide_kernel<FMT, D, NG, WARPS, X, T><<<*grid, 32 * WARPS, Q::SMEM, s>>>(A);
    return cudaGetLastError();
}
// (Trees take the form for capped or biased scores whatever theirs are, and come with bf16 pages or two scales per row.)
template <int FMT, int D, int NG, bool T>
cudaError_t launch_x(const AttnArgs &A, int warps, cudaStream_t s, int *grid)
{
    const bool x = T || A.softcap > 0.0f || A.slopes;
    if constexpr (T && FMT != kBf16 && NG == 1) {
        return cudaErrorInvalidValue;
    } else {
        // nested pages with one scale per row come with at most 32 vectors: more go to the tensor cores
        if constexpr (FMT == kBf16 || NG == 2)
            if (warps == 8) {
                if (x) return launch<FMT, D, NG, 8, true, T>(A, s, grid);
                if constexpr (!T) return launch<FMT, D, NG, 8, false, T>(A, s, grid);
            }
        if (warps != 4) return cudaErrorInvalidValue;
        if (x) return launch<FMT, D, NG, 4, true, T>(A, s, grid);
        if constexpr (!T) return launch<FMT, D, NG, 4, false, T>(A, s, grid);
    }
}
template <int FMT, bool T>
cudaError_t launch_d(const AttnArgs &A, int warps, cudaStream_t s, int *grid)
{
    if (A.p.D == 64) return launch_x<FMT, 64, 1, T>(A, warps, s, grid);
    if constexpr (FMT != kBf16)
        if (A.p.NG == 2) return launch_x<FMT, 128, 2, T>(A, warps, s, grid);
    return launch_x<FMT, 128, 1, T>(A, warps, s, grid);
}

}  // namespace
}  // namespace nq
