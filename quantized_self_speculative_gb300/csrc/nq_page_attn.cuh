// nq_page_attn.cuh -- what the three attention kernels over the paged cache share:
// the list of steps and its runs, the ring of bulk copies, small arithmetic.
#pragma once

#include "nq_mbar.cuh"
#include "nq_page.cuh"

namespace nq {

enum { kBf16 = 0, kKv4 = 1, kKv8 = 2 };

constexpr float kLog2e = 1.4426950408889634f;
// m is raised to 2^lead below the maximum, and only when the largest P = 2^(s - m) has
// passed 2^slack, so that the accumulators are rarely rescaled: a factor of 2^12 in
// between (at 2^6 some row of 32 outgrew it at nearly every step of 64 keys).  fp16
// holds P <= 2^15, and below its normal part rounds by 2^-25: 2^-28 of the maximum at
// most, so that the numerator keeps the tails that the sum of the unrounded P counts
// (n rows: n 2^-28 of it at most; n 2^-23 where trees' V holds its scales, see kSpan
// there).  bf16 has the range of fp32 and rounds P to 2^-8: there the largest P stays 1,
// which is exact.
template <int FMT> __host__ __device__ constexpr float lead() { return FMT == kBf16 ? 0.0f : 3.0f; }
template <int FMT> __host__ __device__ constexpr float slack() { return FMT == kBf16 ? 0.0f : 15.0f; }

struct AttnArgs {
    Pool p;
    Map m;
    const __nv_bfloat16 *q;
    long long q_stride;
    int B, M, Hq, G, QT, cols;          // G query heads per kv head, QT tiles of cols vectors per (sequence, kv head)
    unsigned g_mul;                     // ceil(2^32 / G)
    const int32_t *seqs, *len;
    float scale, softcap;
    int window;
    const float *slopes;
    __nv_bfloat16 *out;
    int4 *info;                         // per CTA: the segment it leaves to later CTAs; x = -1: none, or it gave up
    float *part_o, *part_ml;
    unsigned int *status;
    unsigned long long wait_ns;         // limit of a wait on a barrier
    int starve;                         // steps after which each feed stops (a diagnostic); -1: none
    const uint32_t *tree_bits;          // trees (the kernels' T forms): what node m of sequence b sees, and its depth
    const int32_t *tree_depth;
    int tree_words;
};

// Query row of vector v = row * G + head of the group (v, G <= 2^16).
__device__ __forceinline__ int row_of_vector(const AttnArgs &A, int v) { return A.G == 1 ? v : __umulhi(v, A.g_mul); }

// More than 16 query vectors per kv head: tiles of A.cols columns, *grid CTAs.
cudaError_t attn_wide(int fmt, const AttnArgs &A, cudaStream_t s, int *grid);   // nq_page_attn_wide.cu, 32 or 64
cudaError_t attn_tc(int fmt, const AttnArgs &A, cudaStream_t s, int *grid);     // nq_page_attn_tc.cu, up to 128
// Trees: the T forms of the first two, and a tensor-core kernel of their own.
cudaError_t attn_tree(int fmt, const AttnArgs &A, cudaStream_t s, int *grid);        // nq_page_attn_tree.cu, 8 or 16
cudaError_t attn_tree_wide(int fmt, const AttnArgs &A, cudaStream_t s, int *grid);   // nq_page_attn_tree_wide.cu, 32 or 64
cudaError_t attn_tree_tc(int fmt, const AttnArgs &A, cudaStream_t s, int *grid);     // nq_page_attn_tree_tc.cu, up to 256
// Bytes of a block of 16 rows: base (or bf16), and refinement where it is read.
__host__ __device__ constexpr int block_base(int fmt, int D, int NG) { return fmt == kBf16 ? 64 * D : 16 * D + 64 * NG; }
__host__ __device__ constexpr int block_resid(int fmt, int D) { return fmt == kKv8 ? 16 * D : 0; }

namespace {

// ---------------------------------------------------------------- small pieces
template <int FMT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (FMT == kBf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        mma_f16(d, a0, a1, a2, a3, b0, b1);
}
// the same, from accumulators c
template <int FMT>
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                         float c0, float c1)
{
    if constexpr (FMT == kBf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                     "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_b(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// cap tanh(x / cap), inv = 1 / cap.  With u = x / cap the form 1 - 2 / (1 + e^(2 u)) is
// off by 2^-22 of the cap: little for a score of cap / 8, much for one far below.
// There the Taylor series (relative error 2^-29).
__device__ __forceinline__ float cap_near(float x, float inv)
{
    const float u = x * inv, z = u * u;
    return fmaf(x * z, fmaf(z, fmaf(z, -0.053968254f, 0.13333333f), -0.33333333f), x);
}
__device__ __forceinline__ float cap_far(float x, float cap, float inv)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2(x * (2.0f * kLog2e * inv))));
    return cap * fmaf(-2.0f, r, 1.0f);
}
__device__ __forceinline__ float capped(float x, float cap, float inv)
{
    return fabsf(x) * inv < 0.125f ? cap_near(x, inv) : cap_far(x, cap, inv);
}
// The N scores of one row that a thread holds, those that a mask hides set to 0 before:
// one form for all of them, the error 2^-19 of the largest at most.  (64 scores: 132 us
// against 169 score by score, 36 vectors x 16 sequences; with the four or eight of the
// other kernels it is the other way, 46.8 us against 44.2.)
template <int N>
__device__ __forceinline__ void cap_all(float (&x)[N], float cap, float inv)
{
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(x[i]));
    if (top * inv < 0.125f) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = cap_near(x[i], inv);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = cap_far(x[i], cap, inv);
    }
}
// First row that the query in row `own` sees; no sum passes 32 bits whatever the window.
__device__ __forceinline__ int first_seen(const AttnArgs &A, int own)
{
    return A.window > 0 && own >= A.window ? own - A.window + 1 : 0;
}
// The tree of a sequence of which `base` rows are committed: node j lies in row base + j.
struct TreeOf {
    const uint32_t *bits;
    const int32_t *depth;
    int base, M, words;
    __device__ __forceinline__ TreeOf() {}
    __device__ __forceinline__ TreeOf(const AttnArgs &A, int b, int hi)
        : bits(A.tree_bits + static_cast<size_t>(b) * A.M * A.tree_words), depth(A.tree_depth + static_cast<size_t>(b) * A.M), base(hi - A.M), M(A.M),
          words(A.tree_words)
    {
    }
    __device__ __forceinline__ bool used(int m) const { return depth[m] >= 0; }
    // a row that some node's query may see: one of an unused node may hold anything
    __device__ __forceinline__ bool live(int row) const { return row < base || (row - base < M && used(row - base)); }
    __device__ __forceinline__ int position(int row) const { return row < base || row - base >= M ? row : base + depth[row - base]; }
    // whether node m, at position `own`, sees a row (the window of the nodes is in their bits)
    __device__ __forceinline__ bool sees(int m, int own, int row, unsigned window) const
    {
        const int j = row - base;
        if (j < 0) return static_cast<unsigned>(own - row) < window;
        return j < M && (bits[static_cast<size_t>(m) * words + (j >> 5)] >> (j & 31) & 1u);
    }
};
// max over the eight lanes of a query column, sum likewise
__device__ __forceinline__ float col_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float col_sum(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Nibbles i (low half) and i + 4 (high half) of a word as fp16 halves: KV4
// (q4 + 8) 2^-24, 16 times that for odd i (the other operand or the output
// carries the 1/16); KV8 (16 q4 + r + 136) 2^-24, whose even and odd code bytes
// are formed once per word.
template <int FMT>
struct Codes {
    uint32_t e, o;
    __device__ __forceinline__ Codes(uint32_t b, uint32_t r)
    {
        if constexpr (FMT == kKv8) {
            e = ((b << 4) & 0xF0F0F0F0u) | (r & 0x0F0F0F0Fu);
            o = (b & 0xF0F0F0F0u) | ((r >> 4) & 0x0F0F0F0Fu);
        } else {
            e = b;
            o = b >> 8;
        }
    }
    __device__ __forceinline__ uint32_t pair(int i) const
    {
        if constexpr (FMT == kKv8) {
            const uint32_t x = i & 1 ? o : e;
            return i >= 2 ? __byte_perm(x, 0u, 0x4341) : x & 0x00FF00FFu;
        } else {
            const uint32_t x = i >= 2 ? o : e;
            return i & 1 ? x & 0x00F000F0u : x & 0x000F000Fu;
        }
    }
    // the same pair as signed numbers, q4 or 16 q4 + r, exact
    __device__ __forceinline__ uint32_t value(int i) const
    {
        uint32_t x;
        if constexpr (FMT == kKv8) {
            x = __byte_perm(i & 1 ? o : e, 0x64646464u, i >= 2 ? 0x4341 : 0x4240);               // 1024 + code
            asm("add.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(0xE488E488u));                        // - 1160
        } else {
            x = i >= 2 ? o : e;
            asm("lop3.b32 %0, %0, %1, %2, 0xEA;" : "+r"(x) : "r"(i & 1 ? 0x00F000F0u : 0x000F000Fu), "r"(0x64006400u));   // 1024 + code (16 code)
            if (i & 1) asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(x) : "r"(0x2C002C00u), "r"(0xD480D480u));   // / 16 - 72
            else asm("add.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(0xE408E408u));                   // - 1032
        }
        return x;
    }
};
template <int FMT> __host__ __device__ constexpr float odd_scale() { return FMT == kKv4 ? 16.0f : 1.0f; }

// ---------------------------------------------------------------- sequences
// The rows [lo, hi) of a sequence that any of its queries sees, as steps of SR.
// lo is a multiple of 16 (a block lies in one page), so that no page wholly before
// the window is looked up; steps may begin anywhere in a page.
struct Seq {
    int slot, lo, hi, steps;
};
template <int SR>
__device__ __forceinline__ Seq seq_of(const AttnArgs &A, int b, bool report)
{
    Seq s;
    s.slot = A.seqs ? A.seqs[b] : b;
    const long long cap = min(static_cast<long long>(A.m.W) * A.m.P, 0x7ffff000ll);   // rows of a step past the last one stay in 32 bits
    int n = A.len[b];
    if (n > cap) {
        n = static_cast<int>(cap);
        if (report) set_status(A.status, NQ_DEV_SEQ_FULL);
    }
    if (s.slot < 0 || s.slot >= A.m.S) {
        n = 0;
        s.slot = 0;
        if (report) set_status(A.status, NQ_DEV_BAD_PAGE);
    }
    s.hi = max(n, 0);
    // the first query's own row is hi - M
    s.lo = first_seen(A, s.hi - A.M) / 16 * 16;
    s.steps = s.hi > s.lo ? (s.hi - s.lo + SR - 1) / SR : 0;
    return s;
}

// A position in the flat list: step `at` of segment (b, seg); [begin, end) the
// run's steps of this segment, in flat numbers.
template <int SR>
struct Walk {
    int b, seg;
    Seq s;
    int base, end, stop;                // flat number of the segment's step 0; end of its part; end of the run
    __device__ __forceinline__ void open(const AttnArgs &A, int b0, int b_base, int f0, int f1)
    {
        b = b0;
        s = seq_of<SR>(A, b, false);
        seg = (f0 - b_base) / s.steps;
        base = b_base + seg * s.steps;
        stop = f1;
        end = min(base + s.steps, stop);
    }
    // to the next segment (only called while end < stop)
    __device__ __forceinline__ void next(const AttnArgs &A, int segs)
    {
        base += s.steps;
        if (++seg == segs) {
            seg = 0;
#pragma unroll 1
            do s = seq_of<SR>(A, ++b, false);
            while (s.steps == 0);
        }
        end = min(base + s.steps, stop);
    }
};

// The calling CTA's run [f0, f1) of the flat list: equal runs of at least
// min_run steps, and the sequence in which it starts (its first flat number
// `base`).  Writes the zeros of sequences of which no query sees a row.
struct Run {
    int f0, f1, per, b, base;
};
template <int SR, int THREADS, int D>
__device__ __forceinline__ Run find_run(const AttnArgs &A, int segs, int min_run)
{
    constexpr int WARPS = THREADS / 32;
    __shared__ int sh_sum[WARPS], sh_base, sh_b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_thread = (A.B + THREADS - 1) / THREADS, b_lo = min(static_cast<int>(threadIdx.x) * per_thread, A.B),
              b_hi = min(b_lo + per_thread, A.B);
    int mine = 0;
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) mine += seq_of<SR>(A, b, blockIdx.x == 0).steps * segs;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sh_sum[warp] = incl;
    __syncthreads();
    int total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += sh_sum[w];
        total += sh_sum[w];
    }
    Run r;
    const int grid = gridDim.x;
    r.per = max(total / grid + (total % grid != 0), min_run);
    r.f0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * r.per, static_cast<long long>(total)));
    r.f1 = total - r.f0 < r.per ? total : r.f0 + r.per;
    if (r.f0 < r.f1 && r.f0 >= before && r.f0 < before + mine) {
        int at = before;
#pragma unroll 1
        for (int b = b_lo; b < b_hi; ++b) {
            const int n = seq_of<SR>(A, b, false).steps * segs;
            if (r.f0 < at + n) {
                sh_b = b;
                sh_base = at;
                break;
            }
            at += n;
        }
    }
#pragma unroll 1
    for (int b = blockIdx.x; b < A.B; b += grid) {
        if (seq_of<SR>(A, b, false).steps != 0) continue;
        const size_t n = static_cast<size_t>(A.M) * A.Hq * (D / 8);
        uint4 *o = reinterpret_cast<uint4 *>(A.out) + b * n;
#pragma unroll 1
        for (size_t i = threadIdx.x; i < n; i += THREADS) o[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    r.b = sh_b;
    r.base = sh_base;
    return r;
}

// Fills a ring with the steps f, f + STRIDE, .. of a run: the whole warp walks,
// lane k copies block k of the step (and those that follow it in its page).  The
// page ids of a step are loaded one step ahead.  Blocks of a page outside the pool
// are not copied: `gone` takes their bits, and their rows are masked.
template <int FMT, int D, int NG, int BLKS, int STRIDE>
struct Feed {
    static constexpr int SR = 16 * BLKS, BASE = block_base(FMT, D, NG), RESID = block_resid(FMT, D), STAGE = BLKS * (BASE + RESID);
    Walk<SR> w;
    int row, left, id, lp;                    // row of the next step; how many are left in this segment (0: none at all); lane's page
    const int32_t *tab;
    const uint8_t *rec;
    uint32_t ring, bar;

    __device__ __forceinline__ void aim(const AttnArgs &A, int segs, int f)   // at step f or the first one after it
    {
#pragma unroll 1
        while (f >= w.end) {
            if (w.end >= w.stop) {
                left = 0;
                return;
            }
            w.next(A, segs);
        }
        row = w.s.lo + (f - w.base) * SR;
        left = (w.end - f + STRIDE - 1) / STRIDE;
        tab = A.m.table + static_cast<size_t>(w.s.slot) * A.m.W;
        rec = A.p.data + static_cast<size_t>(w.seg / A.QT) * A.p.rec;
    }
    __device__ __forceinline__ void look()
    {
        const int k = threadIdx.x & 31, r = row + 16 * k;
        if (left > 0 && k < BLKS && r < w.s.hi) id = tab[r >> lp];
    }
    __device__ __forceinline__ void start(const AttnArgs &A, const Walk<SR> &at, int segs, int f, uint32_t ring_, uint32_t bar_)
    {
        w = at;
        if (A.starve >= 0) {
            w.stop = static_cast<int>(min(static_cast<long long>(w.stop), f + static_cast<long long>(A.starve) * STRIDE));
            w.end = min(w.end, w.stop);
        }
        ring = ring_;
        bar = bar_;
        lp = 31 - __clz(A.m.P);
        id = 0;
        aim(A, segs, f);
        look();
    }
    template <typename F>
    __device__ __forceinline__ void issue(const AttnArgs &A, int segs, int st, F gone)   // the step into stage st, then on to the next
    {
        if (left == 0) return;
        const int k = threadIdx.x & 31, n = min(BLKS, (w.s.hi - row + 15) >> 4), blk = ((row + 16 * k) & (A.m.P - 1)) >> 4;
        const uint32_t b = bar + 8 * st, dst = ring + st * STAGE;
        const bool bad = k < n && (id < 0 || id >= A.p.N);
        const uint32_t out = __ballot_sync(0xffffffffu, bad);
        gone(out);
        if (k == 0) mbar_expect_tx(b, (n - __popc(out)) * (BASE + RESID));
        __syncwarp();
        if (bad) {
            set_status(A.status, NQ_DEV_BAD_PAGE);
        } else if (k < n && (k == 0 || blk == 0)) {
            const int x = min(n - k, (1 << (lp - 4)) - blk);                     // blocks side by side in the page
            const uint8_t *src = rec + static_cast<size_t>(id) * A.p.H * A.p.rec;
            bulk_g2s(dst + k * BASE, src + blk * BASE, x * BASE, b);
            if constexpr (FMT == kKv8) bulk_g2s(dst + BLKS * BASE + k * RESID, src + A.p.resid_off + blk * RESID, x * RESID, b);
        }
        __syncwarp();
        row += STRIDE * SR;
        if (--left == 0) aim(A, segs, w.base + (row - w.s.lo) / SR);
        look();
    }
    // Waits for stage st, of a ring in which `filled` hold or await a step.  Where that gives
    // up, nothing more is issued: the CTA goes on to the end of its run without waiting.
    __device__ __forceinline__ void wait(const AttnArgs &A, uint32_t bar_, int st, uint32_t phase, int stages, int &filled, int *abort_flag)
    {
        if (!ring_wait(bar_, st, phase, filled, stages, abort_flag, A.status, A.wait_ns)) left = filled = 0;
    }
};

}  // namespace
}  // namespace nq
