// nq_page_attn_tree_tc.cu -- attention of trees over nested pages for many query
// vectors per kv head, on the 5th-generation tensor cores.
//
// A tree of 32 nodes with four query heads per kv head is 128 query vectors, of 64
// nodes with seven 448: products, softmax and decoding bound the time, not HBM.  As
// in nq_page_attn_tc.cu a row of the tensor cores is a query vector and a step is 64
// cache rows, decoded once: K into signed fp16 codes (exact; its scales multiply S), V
// into fp16 values relative to a power of two 2^E near the step's largest scale (one
// rounding, 2^-11; P carries the 2^E).  Where a step's scales span more than 2^4 (kSpan) or
// one of them is 0, and where it has rows that some query does not see, V stays codes, and
// its scales multiply P.
// That leaves the softmax one scale per key to read: with V's scale and its log2 as
// well shared memory is 77% busy (13 instead of 19 million wavefronts, the long case
// below).  One warp per scheduler does not fill the softmax's dependent chain
// (load S, scale, maximum, exp2, store P: some 1700 cycles for 64 keys), so that here
// two groups of four softmax warps work at once:
//   KS = false (129 .. 256 vectors): group g has vectors 128 g .. of the tile, both take
//     every step, which is decoded once for 256 vectors.
//   KS = true (up to 128 vectors): both have the same vectors, group g takes the steps
//     g, g + 2, .. with a state of its own; group 0 merges the two at a segment's end
//     (row r of both accumulators lies in the same lane of tensor memory).
// Q lies in shared memory.  S is double-buffered per group, and P takes the place of
// its S.  V needs no transpose: its rows along N are an MN-major operand.
//
// Warp roles, handing on through mbarriers (all waits bounded):
//   0-7   softmax: group w / 4, lane quarter w % 4 of tensor memory; also Q in, O out
//   8-15  decode: stage -> K, V, scales
//   16-17 issue the MMAs of group 0, 1: S one of the group's steps ahead of its P V.  (A warp's issue waits while the
//         tensor pipe works: 460 cycles for S, 260 for P V; one warp for both groups is late for every step.)
//   18-19 feed the ring of raw blocks, every second step each
// Partial states and join as in the other kernels; one CTA per SM; runs are equal in
// cost, of which a segment's begin and end are eight steps' worth.
//
// Measured (GB300, 8-bit view): 16 sequences of 333..4131 rows, 8 kv heads of 128, trees
// of up to 32 nodes, 128 vectors: 55 us for 86 MB and 20 GFLOP (13 us at the copy rate; the
// warp-MMA kernels 233); 4 of 20065..32832 rows, 4 kv heads, 64 nodes x 7 heads: 137 us
// for 104 GFLOP (55 us at the measured bf16 rate, 40%; the warp-MMA kernels 988).  A step
// of 256 vectors takes some 2400 cycles: the tensor pipe 1020, the softmax of a group 1600
// beside some 800 of waits, fences and loop.  All forms spill (40 to 80 bytes of
// stores per thread, 92 to 312 of loads; under a cap or bias 216 to 224 and 300 to 348).  A cap
// doubles the time: 16 sequences of 500..4000 rows, 8 kv heads of 128, 36 / 128 / 256 vectors,
// plain 51 / 55 / 72 us, capped 101 / 114 / 176, with a bias too 121 / 131 / 222.
#include <atomic>

#include "nq_page_attn.cuh"
#include "nq_tcgen.cuh"

namespace nq {
namespace {

constexpr int kGroups = 2, kGroupWarps = 4, kSoftWarps = kGroups * kGroupWarps, kDecodeWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kDecodeWarps, kFeedWarp = kMmaWarp + kGroups, kFeedWarps = 2;
constexpr int kThreads = 20 * 32;       // five warps per scheduler, whole warpgroups
static_assert(kThreads == 32 * (kFeedWarp + kFeedWarps), "roles");
// Registers per thread: launched with 96 each, from which the warpgroups' shares are drawn.
constexpr int kRegsLaunch = 96, kRegsSoft = 128, kRegsDecode = 72, kRegsRest = 80;
static_assert(2 * kRegsSoft + 2 * kRegsDecode + kRegsRest == 5 * kRegsLaunch, "setmaxnreg draws on the launch's registers");
constexpr int kMinRun = 2;              // steps per CTA
// What a segment costs beside its steps, in steps.  us with 4 / 6 / 8 / 12, 16 sequences of 500..4000 rows, 8 kv heads:
// heads of 128, 20 vectors 54 / 50 / 49 / 50, 128 vectors 60 / 55 / 55 / 54, 256 vectors 76 / 72 / 72 / 74; heads of 64,
// 128 vectors 46 / 43 / 43 / 43, 256 vectors 64 / 66 / 68 / 71 (the one form that 4 suits better).
constexpr int kSegCost = 8;
constexpr int kKeys = 64;               // cache rows per step
constexpr int kTmem = 512;              // columns: S (P) of group g, buffer b at 64 (2 g + b), O of group g at 256 + 128 g
constexpr uint32_t kColO = 256;
constexpr int kCodes = 1000;
// V's scales of a step may span 2^kSpan where they go into its values.  P is then relative to the step's largest scale, not
// to each row's: of a largest contribution from a row with the smallest scale the reference lies up to 2^(kSpan + 1) above
// it, and P's rounding of 2^-25 below fp16's normal numbers is 2^(kSpan - 27) of it, n rows' n times that (2^-28 among codes).
// At 12, where V itself would leave the normal numbers, 12000 rows below one key with nearly all the weight and a value
// 2^11 below theirs were lost, some hundredths of the output.
constexpr int kSpan = 4;
constexpr uint32_t kHidden = 0x100;      // with the bits of the blocks that are not there: the step has rows that some query does not see

template <int FMT, int D, bool KS>
struct Tt {
    static constexpr int BASE = block_base(FMT, D, 1), RESID = block_resid(FMT, D);
    static constexpr int BLKS = kKeys / 16, STAGE = BLKS * (BASE + RESID);
    static constexpr int Q_BYTES = 128 * D * 2, Q_TILES = KS ? 1 : 2;
    static constexpr int K_BYTES = kKeys * D * 2, PANEL = kKeys * 128;       // 64 dimensions of 64 rows
    static constexpr int BUF = 2 * K_BYTES;                                  // K, V of one step
    static constexpr int SCALES = 3 * kKeys * 4;                             // K's, V's, log2 of V's
    static constexpr int BUFS = KS ? 4 : 3;                                  // decoded steps
    static constexpr int STAGES = 3;
    static constexpr int SMEM = Q_TILES * Q_BYTES + BUFS * (BUF + SCALES) + STAGES * STAGE;
    static_assert(SMEM <= 227 * 1024 - 2048, "shared memory");
};

// Barriers by number.
constexpr int kRawFull = 0, kRawEmpty = 4, kKvFull = 8, kKvEmpty = 12, kSFull = 16, kPFull = 20, kPvDone = 24, kQFull = 28, kState = 29, kDrain = 30,
              kBars = 32;

// Bits of the 32 rows from `row` on that node m of the tree sees, at position `own`; rows in front of a window that
// ends at `from` are hidden among the committed ones (the nodes' own bits hold the window).
__device__ __forceinline__ uint32_t seen32(const TreeOf &t, int m, int from, int row)
{
    const int j = row - t.base, w = j >> 5;                      // w = -1: the border of the committed rows lies in the word
    if (j <= -32) return from <= row ? 0xffffffffu : from >= row + 32 ? 0u : 0xffffffffu << (from - row);
    const uint32_t *b = t.bits + static_cast<size_t>(m) * t.words;
    const uint32_t lo = w < 0 ? 0xffffffffu : w < t.words ? b[w] : 0u, hi = w + 1 < t.words ? b[w + 1] : 0u;
    uint32_t x = __funnelshift_r(lo, hi, j & 31);
    const int cut = min(from, t.base) - row;                     // committed rows before the window
    if (cut > 0) x &= cut >= 32 ? 0u : 0xffffffffu << cut;
    return x;
}

// Where a step's blocks lie in a stage: base block j at j step, its refinement at j
// rstep + roff.  A page of 16 rows is one run of bytes, its base block and its
// refinement, and comes by one copy; larger pages bring all base blocks, then all
// refinements.
template <int FMT, int D>
struct Place {
    int step, roff, rstep;
    __device__ __forceinline__ explicit Place(const AttnArgs &A)
    {
        constexpr int BASE = block_base(FMT, D, 1), RESID = block_resid(FMT, D);
        const bool one = FMT == kKv8 && A.p.P == 16;
        step = one ? BASE + RESID : BASE;
        roff = one ? BASE : kKeys / 16 * BASE;
        rstep = one ? BASE + RESID : RESID;
    }
};
// The feed of the other kernels costs its warp some 2000 cycles a step of eight copies:
// each waits for the step's page ids, and takes some 190 where its operands are not
// provably uniform.  Here lane l holds the page of block l of the 32 blocks from
// `base` on, and of the 32 after them, and the copies go out from shuffled operands.
template <int FMT, int D>
struct Feeder {
    static constexpr int BLKS = kKeys / 16, BASE = block_base(FMT, D, 1), RESID = block_resid(FMT, D), STAGE = BLKS * (BASE + RESID);
    Walk<kKeys> w;
    int row, left, base, id, id_next, lp;     // row of the next step; how many are left in this segment (0: none at all)
    const int32_t *tab;
    const uint8_t *rec;
    uint32_t ring, bar;

    __device__ __forceinline__ int page_of(int from) const
    {
        const int r = from + 16 * (threadIdx.x & 31);
        return r >= from && r < w.s.hi ? tab[r >> lp] : 0;       // (r past 2^31 is below `from`)
    }
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
        row = base = w.s.lo + (f - w.base) * kKeys;
        left = (w.end - f + kFeedWarps - 1) / kFeedWarps;
        tab = A.m.table + static_cast<size_t>(w.s.slot) * A.m.W;
        rec = A.p.data + static_cast<size_t>(w.seg / A.QT) * A.p.rec;
        id = page_of(base);
        id_next = base < 0x7ffffe00 - 512 ? page_of(base + 512) : 0;
    }
    __device__ __forceinline__ void start(const AttnArgs &A, const Walk<kKeys> &at, int segs, int f, uint32_t ring_, uint32_t bar_)
    {
        w = at;
        ring = ring_;
        bar = bar_;
        lp = 31 - __clz(A.m.P);
        aim(A, segs, f);
    }
    // The step into stage st, then on to the next; gone takes the blocks that are not there, of pages outside the pool.
    __device__ __forceinline__ void issue(const AttnArgs &A, const Place<FMT, D> &at, int segs, int st, uint32_t &gone)
    {
        const int k = threadIdx.x & 31, n = min(BLKS, (w.s.hi - row + 15) >> 4), blk = ((row + 16 * k) & (A.m.P - 1)) >> 4;
        const int mine = __shfl_sync(0xffffffffu, id, ((row - base) >> 4) + (k & (BLKS - 1)));
        const uint32_t b = bar + 8 * st, dst = ring + st * STAGE;
        const bool bad = k < n && (mine < 0 || mine >= A.p.N);
        const uint32_t out = __ballot_sync(0xffffffffu, bad);
        if (bad) set_status(A.status, NQ_DEV_BAD_PAGE);
        // before the barrier's arrival, which lets the decoders read it.  Where some row is hidden from some query nothing
        // may depend on what such rows hold (or what a stage held before): V stays codes there
        const bool masked = row < first_seen(A, w.s.hi - 1) || row + kKeys > w.s.hi - A.M;
        gone = out | (masked ? kHidden : 0u);
        __syncwarp();
        if (k == 0) mbar_expect_tx(b, (n - __popc(out)) * (BASE + RESID));
        __syncwarp();
#pragma unroll 1
        for (uint32_t todo = __ballot_sync(0xffffffffu, !bad && k < n && (k == 0 || blk == 0)); todo; todo &= todo - 1) {
            const int j = __ffs(todo) - 1, jb = __shfl_sync(0xffffffffu, blk, j), x = min(n - j, (1 << (lp - 4)) - jb);   // blocks side by side in the page
            const uint8_t *src = rec + static_cast<size_t>(__shfl_sync(0xffffffffu, mine, j)) * A.p.H * A.p.rec;
            if (elect_one()) {
                bulk_g2s(dst + j * at.step, src + jb * BASE, x * at.step, b);    // (x = 1 where the step holds the refinement too)
                if (FMT == kKv8 && at.step == BASE) bulk_g2s(dst + at.roff + j * at.rstep, src + A.p.resid_off + jb * RESID, x * RESID, b);
            }
            __syncwarp();
        }
        row += kFeedWarps * kKeys;
        if (--left == 0) {
            aim(A, segs, w.base + (row - w.s.lo) / kKeys);
        } else if (row - base >= 512) {
            base += 512;
            id = id_next;
            id_next = base < 0x7ffffe00 - 512 ? page_of(base + 512) : 0;
        }
    }
};

// As find_run, but a segment's begin and end (queries in, rows out, pipelines that fill and
// drain) count as kSegCost steps before its first: of ragged sequences some CTAs would
// otherwise have five short segments where others have a part of one, and take twice as long.
// f0, f1 are flat numbers of steps; `per` counts costs, of which segment number `seg`
// (among all that have steps) begins at its flat number + seg * kSegCost.
struct CostRun {
    int f0, f1, per, b, base, seg;
};
template <int SR, int THREADS, int D>
__device__ __forceinline__ CostRun find_cost_run(const AttnArgs &A, int segs)
{
    constexpr int WARPS = THREADS / 32;
    __shared__ int2 sh_sum[WARPS];
    __shared__ int sh_f[2], sh_b, sh_base, sh_seg;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_thread = (A.B + THREADS - 1) / THREADS, b_lo = min(static_cast<int>(threadIdx.x) * per_thread, A.B),
              b_hi = min(b_lo + per_thread, A.B);
    int2 mine = make_int2(0, 0);              // steps, segments
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) {
        const int n = seq_of<SR>(A, b, blockIdx.x == 0).steps;
        mine.x += n * segs;
        mine.y += n ? segs : 0;
    }
    int2 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
        if (lane >= o) {
            incl.x += x;
            incl.y += y;
        }
    }
    if (lane == 31) sh_sum[warp] = incl;
    __syncthreads();
    int2 total = make_int2(0, 0), before = make_int2(incl.x - mine.x, incl.y - mine.y);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) {
            before.x += sh_sum[w].x;
            before.y += sh_sum[w].y;
        }
        total.x += sh_sum[w].x;
        total.y += sh_sum[w].y;
    }
    if (threadIdx.x < 2) sh_f[threadIdx.x] = total.x;            // (an end past the last cost)
    __syncthreads();
    CostRun r;
    const int all = total.x + kSegCost * total.y, grid = gridDim.x;
    r.per = max(all / grid + (all % grid != 0), kMinRun + kSegCost);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {                       // the run's first cost, and that of the next run
        const long long c = static_cast<long long>(blockIdx.x + side) * r.per;
        long long at = before.x + static_cast<long long>(kSegCost) * before.y;
        if (c < at || c >= at + mine.x + static_cast<long long>(kSegCost) * mine.y) continue;
        int flat = before.x, seg = before.y;
#pragma unroll 1
        for (int b = b_lo; b < b_hi; ++b) {
            const int n = seq_of<SR>(A, b, false).steps;
            if (n == 0) continue;
            const long long cost = static_cast<long long>(n + kSegCost) * segs;
            if (c < at + cost) {
                const int k = static_cast<int>((c - at) / (n + kSegCost)), off = static_cast<int>(c - at) - k * (n + kSegCost);
                sh_f[side] = flat + k * n + max(off - kSegCost, 0);
                if (side == 0) {
                    sh_b = b;
                    sh_base = flat;
                    sh_seg = seg + k;
                }
                break;
            }
            at += cost;
            flat += n * segs;
            seg += segs;
        }
    }
#pragma unroll 1
    for (int b = blockIdx.x; b < A.B; b += grid) {               // zeros of sequences of which no query sees a row
        if (seq_of<SR>(A, b, false).steps != 0) continue;
        const size_t n = static_cast<size_t>(A.M) * A.Hq * (D / 8);
        uint4 *o = reinterpret_cast<uint4 *>(A.out) + b * n;
#pragma unroll 1
        for (size_t i = threadIdx.x; i < n; i += THREADS) o[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    r.f0 = sh_f[0];
    r.f1 = sh_f[1];
    r.b = sh_b;
    r.base = sh_base;
    r.seg = sh_seg;
    return r;
}
// mbar_wait_fast without its call: with one in it ptxas does not allocate a warpgroup's own share of registers.
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, volatile int *abort_flag, unsigned int *status, unsigned long long limit_ns)
{
#pragma unroll 1
    for (int i = 0; i < 256; ++i) {
        uint32_t ok;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (ok) return true;
    }
    const unsigned long long t0 = global_ns();
#pragma unroll 1
    while (!mbar_try(bar, parity)) {
        if (*abort_flag) return false;
        if (global_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            set_status(status, NQ_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
// A value that is the same on all lanes, so that the compiler knows it: what tcgen05.mma takes lies in uniform registers, and
// an operand that it cannot prove uniform costs some 190 cycles per MMA instead of 34 to 66.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

template <int FMT, int D, bool X, bool KS>
__global__ void __launch_bounds__(kThreads, 1)
attn_tree_tc_kernel(const __grid_constant__ AttnArgs A)
{
    using Q = Tt<FMT, D, KS>;
    constexpr int SR = kKeys, RB = D / 2, STRIDE = KS ? kGroups : 1;            // of a group's steps
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ __align__(8) unsigned long long bars[kBars];
    __shared__ uint32_t gone_of[Q::STAGES];                                      // blocks that are not there
    __shared__ int2 about[Q::BUFS];                                              // the same; E of V's values, kCodes: they are codes
    __shared__ float2 state[KS ? 128 : 1];                                       // of group 1, for group 0
    __shared__ float cq_of[Q::Q_TILES * 128];                                    // factor of a query's scores
    __shared__ int abort_flag, keep_tmem;
    __shared__ uint32_t tmem_slot;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
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
            mbar_init(bar(kKvEmpty + i), KS ? 1 : kGroups);
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kPFull + i), kGroupWarps);
            mbar_init(bar(kPvDone + i), 1);
        }
        mbar_init(bar(kQFull), KS ? kGroupWarps : kSoftWarps);
        mbar_init(bar(kState), kGroupWarps + 1);
        for (int g = 0; g < kGroups; ++g) mbar_init(bar(kDrain + g), 32);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const CostRun run = find_cost_run<SR, kThreads, D>(A, segs);
    if (run.f0 >= run.f1) return;
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(kTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(tmem_slot);
    unsigned char *bufs = sm + Q::Q_TILES * Q::Q_BYTES, *scales = bufs + Q::BUFS * Q::BUF, *ring = scales + Q::BUFS * Q::SCALES;
    auto wait = [&](int i, int phase) { return wait_here(bar(i), static_cast<uint32_t>(phase) & 1u, &abort_flag, A.status, A.wait_ns); };
    const int steps = uniform(run.f1 - run.f0);
    Walk<SR> use;
    use.open(A, run.b, run.base, run.f0, run.f1);

    const Place<FMT, D> place(A);
    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp >= kFeedWarp) {
        // ================================================= raw blocks into the ring: every second step
        Feeder<FMT, D> feed;
        int i = warp - kFeedWarp;
        const int fed = A.starve < 0 ? steps : static_cast<int>(min(static_cast<long long>(steps), i + static_cast<long long>(A.starve) * kFeedWarps));
        feed.start(A, use, segs, run.f0 + i, smem_u32(ring), bar(kRawFull));
        for (; i < fed; i += kFeedWarps) {
            const int st = i % Q::STAGES;
            if (!__all_sync(0xffffffffu, wait(kRawEmpty + st, (i / Q::STAGES & 1) ^ 1))) break;
            feed.issue(A, place, segs, st, gone_of[st]);
        }
        // every copy issued has landed before the CTA may exit: the last steps', as the others' stages have been read.  (Where
        // a wait gave up, or the feed stops early: this warp's last two.)
        volatile int never = 0;
        for (int k = i < steps ? i - 2 * kFeedWarps : i - kFeedWarps * Q::STAGES; k < i && k < steps; k += kFeedWarps)
            if (k >= 0 && (i < steps || k >= steps - Q::STAGES)) wait_here(bar(kRawFull + k % Q::STAGES), k / Q::STAGES & 1, &never, A.status, A.wait_ns);
    } else {
        // ================================================= MMAs of group g
        const int g = warp - kMmaWarp;
        const uint32_t idesc_s = f16_idesc(128, kKeys), idesc_o = f16_idesc(128, D) | kMajorMN_B, ts = tmem + 128 * g, to = tmem + kColO + 128 * g;
        const uint64_t q_desc = sw128_desc(smem_u32(sm) + (KS ? 0 : g * Q::Q_BYTES)), k_desc = sw128_desc(smem_u32(bufs)),
                       v_desc = sw128_desc_mn(smem_u32(bufs) + Q::K_BYTES, Q::PANEL);
        uint32_t issued_by = 0, leader;
        int ns = 0, np = 0;                                      // S and P V products issued
        int i0 = 0, seg_no = 0;                                  // first step of the segment (part), in steps of the run
        bool ok = true;
        while (ok && i0 < steps) {
            const int n = uniform(use.end - max(use.base, run.f0));   // its steps; the group's: from g on, every second (KS), or all
            ok = __all_sync(0xffffffffu, wait(kQFull, seg_no));
            if (KS && g == 1 && lane == 0) mbar_arrive(bar(kState));  // so that no barrier gets two phases ahead of a warp without steps
            const int k0 = KS ? g : 0;
            auto scores = [&](int k) {
                const int buf = uniform((i0 + k) % Q::BUFS), b = uniform(ns & 1);
                // decoded, and the buffer's P of two steps ago used
                if (!__all_sync(0xffffffffu, wait(kKvFull + buf, (i0 + k) / Q::BUFS) && (ns < 2 || wait(kPvDone + 2 * g + b, (ns - 2) >> 1)))) return false;
                tc_fence_after();
                // 16 dimensions on: 32 bytes, or the next panel of 64 (descriptors count in 16 bytes)
                const uint64_t kt = k_desc + static_cast<uint32_t>(buf * (Q::BUF >> 4));
                if (elect_one(leader)) {
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
                        tc_mma_ss(ts + 64 * b, q_desc + (d >> 2) * (128 * 128 >> 4) + (d & 3) * 2, kt + (d >> 2) * (Q::PANEL >> 4) + (d & 3) * 2, idesc_s, d != 0);
                    tc_commit(bar(kSFull + 2 * g + b));
                }
                __syncwarp();
                issued_by |= 1u << leader;
                ++ns;
                return true;
            };
            if (ok && k0 < n) ok = scores(k0);
            for (int k = k0; ok && k < n; k += STRIDE) {
                if (k + STRIDE < n) ok = scores(k + STRIDE);
                const int buf = uniform((i0 + k) % Q::BUFS), b = uniform(np & 1);
                ok = ok && __all_sync(0xffffffffu, wait(kPFull + 2 * g + b, np >> 1));
                if (!ok) break;
                tc_fence_after();
                const uint64_t vt = v_desc + static_cast<uint32_t>(buf * (Q::BUF >> 4));
                const uint32_t more = uniform(k != k0);
                if (elect_one(leader)) {
#pragma unroll
                    for (int d = 0; d < kKeys / 16; ++d) tc_mma(to, ts + 64 * b + 8 * d, vt + d * (2048 >> 4), idesc_o, d != 0 ? 1u : more);
                    tc_commit(bar(kPvDone + 2 * g + b));
                    tc_commit(bar(kKvEmpty + buf));
                }
                __syncwarp();
                issued_by |= 1u << leader;
                ++np;
            }
            i0 += n;
            ++seg_no;
            if (i0 < steps) use.next(A, segs);
        }
        // every MMA has completed before tensor memory is freed, whatever ended the loop
        if (issued_by) {
            if ((issued_by >> lane) & 1u) tc_commit(bar(kDrain + g));
            else mbar_arrive(bar(kDrain + g));
            __syncwarp();
            volatile int never = 0;
            const bool drained = wait_here(bar(kDrain + g), 0, &never, A.status, A.wait_ns);
            if (!__all_sync(0xffffffffu, drained) && lane == 0) keep_tmem = 1;
        }
    }
    } else if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecode));
        // ================================================= decode
        const int dt = threadIdx.x - 32 * kSoftWarps;
        for (int i = 0; i < steps; ++i) {
            const int st = i % Q::STAGES, b = i % Q::BUFS;
            if (!__all_sync(0xffffffffu, wait(kRawFull + st, i / Q::STAGES & 1) && wait(kKvEmpty + b, (i / Q::BUFS & 1) ^ 1))) break;
            const unsigned char *sp = ring + st * Q::STAGE;
            unsigned char *buf = bufs + b * Q::BUF;
            // thread = (K or V, row, 16-byte chunk of nibbles): four words of eight values, in the order 0 4 1 5 2 6 3 7
            // that the masks give (Q's columns follow it, and O's are put back)
            constexpr int CH = RB / 16, ALL = 2 * kKeys * CH, N = (ALL + 32 * kDecodeWarps - 1) / (32 * kDecodeWarps);   // CH: 4 (D = 128) or 2
            uint4 xs[N], ys[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int e = dt + k * 32 * kDecodeWarps, v = e / (kKeys * CH), r = e / CH % kKeys, c = e % CH, at = v * 16 * RB + nib_off(RB, r & 15, 16 * c);
                if (e < ALL) {
                    xs[k] = *reinterpret_cast<const uint4 *>(sp + (r >> 4) * place.step + at);
                    if constexpr (FMT == kKv8) ys[k] = *reinterpret_cast<const uint4 *>(sp + place.roff + (r >> 4) * place.rstep + at);
                }
            }
            // a scale that is not finite, or negative, counts as 0: rows that no query sees may hold anything
            auto scale_of = [&](int r, int v) -> uint32_t {
                const uint32_t x = reinterpret_cast<const uint16_t *>(sp + (r >> 4) * place.step + 32 * RB)[16 * v + (r & 15)];
                return x < 0x7C00u ? x : 0u;
            };
            auto number = [](uint32_t x) { return __half2float(__ushort_as_half(static_cast<unsigned short>(x))); };
            const uint32_t s0 = scale_of(lane, 1), s1 = scale_of(lane + 32, 1);
            const uint32_t top = __reduce_max_sync(0xffffffffu, max(s0, s1)), low = __reduce_min_sync(0xffffffffu, min(s0, s1));
            auto exponent = [&](uint32_t x) { return static_cast<int>(__float_as_uint(number(x)) >> 23) - 127; };
            const uint32_t flags = gone_of[st];
            // (a row of scale 0 adds nothing to the numerator: among codes its log2 keeps its score from raising the reference)
            const int E = flags || low == 0 || exponent(top) - exponent(low) > kSpan ? kCodes : exponent(top);
            const float by = __uint_as_float(static_cast<uint32_t>(127 - (E == kCodes ? 0 : E)) << 23);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int e = dt + k * 32 * kDecodeWarps, v = e / (kKeys * CH), r = e / CH % kKeys, c = e % CH;
                if (e >= ALL) break;
                const uint4 x = xs[k], y = FMT == kKv8 ? ys[k] : make_uint4(0, 0, 0, 0);
                // chunks of the upper 64 dimensions in another order: then eight lanes write to eight banks
                const bool swap = c >= 2;
                const uint32_t xw[4] = {swap ? x.z : x.x, swap ? x.w : x.y, swap ? x.x : x.z, swap ? x.y : x.w};
                const uint32_t yw[4] = {swap ? y.z : y.x, swap ? y.w : y.y, swap ? y.x : y.z, swap ? y.y : y.w};
                unsigned char *to = buf + v * Q::K_BYTES + (c >> 1) * Q::PANEL + r * 128;
                const float one = v == 0 || E == kCodes ? 1.0f : number(scale_of(r, 1)) * by;    // exact in fp16
                const uint32_t f2 = pack_h(one, one);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const Codes<FMT> q(xw[w], yw[w]);
                    const int chunk = 4 * (c & 1) + (swap ? w ^ 2 : w);
                    uint32_t d[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d[u]) : "r"(q.value(u)), "r"(f2));
                    *reinterpret_cast<uint4 *>(to + ((chunk ^ (r & 7)) << 4)) = make_uint4(d[0], d[1], d[2], d[3]);
                }
            }
            if (dt < kKeys) {
                float *f = reinterpret_cast<float *>(scales + b * Q::SCALES);
                if (dt == 0) about[b] = make_int2(flags & (kHidden - 1), E);
                f[dt] = number(scale_of(dt, 0));
                if (E == kCodes) {
                    const float sv = number(scale_of(dt, 1));
                    f[kKeys + dt] = sv;
                    f[2 * kKeys + dt] = lg2(fmaxf(sv, 3.7252902984619140625e-09f));              // a scale of 0 has codes of 0
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMAs read, and the next copy writes, through the async proxy
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kKvFull + b));
                mbar_arrive(bar(kRawEmpty + st));
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        // ================================================= softmax: thread = query vector
        const int g = warp >> 2, r = (warp & 3) * 32 + lane, row = KS ? r : 128 * g + r;      // row of the tensor cores; vector of the tile
        const uint32_t tq = tmem + (static_cast<uint32_t>(warp & 3) << 21), to = tq + kColO + 128 * g;
        const float cap2 = A.softcap * kLog2e, inv2 = X && A.softcap > 0.0f ? 1.0f / cap2 : 0.0f;
        int cnt = 0, i0 = 0, seg_no = 0;                         // the group's steps so far; the segment's first step
        auto segment = [&]() {                                   // false where a wait gave up
            const int n = use.end - max(use.base, run.f0);
            const int kvh = use.seg / A.QT, v0 = (use.seg - kvh * A.QT) * A.cols, nv = min(A.cols, A.M * A.G - v0);
            const bool active = (row & ~31) < nv, valid = row < nv;
            const int v = v0 + (valid ? row : nv - 1), m = row_of_vector(A, v), hq = kvh * A.G + v - m * A.G;
            const TreeOf tree(A, use.b, use.s.hi);
            const bool used = tree.used(m);
            const int own = tree.base + tree.depth[m], from = first_seen(A, own);
            // ---- the warp's query rows into shared memory: 16-byte chunks, neighbouring lanes in a row
            if (active && (!KS || g == 0)) {
                constexpr int CH = D / 8, RPI = 32 / CH, N = 32 / RPI;           // chunks per row, rows per load
                const int c = lane % CH;
                uint4 x[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int vk = (row & ~31) + k * RPI + lane / CH, mk = row_of_vector(A, v0 + vk);
                    x[k] = make_uint4(0, 0, 0, 0);
                    if (vk < nv)
                        x[k] = *reinterpret_cast<const uint4 *>(A.q + (static_cast<long long>(use.b) * A.M + mk) * A.q_stride +
                                                                (kvh * A.G + v0 + vk - mk * A.G) * D + 8 * c);
                }
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int rk = (r & ~31) + k * RPI + lane / CH;
                    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                    float f[8], top = 0.0f;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        f[2 * u] = __uint_as_float(w[u] << 16);
                        f[2 * u + 1] = __uint_as_float(w[u] & 0xFFFF0000u);
                        top = fmaxf(top, fmaxf(fabsf(f[2 * u]), fabsf(f[2 * u + 1])));
                    }
#pragma unroll
                    for (int o = 1; o < CH; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // largest magnitude to [2^10, 2^11) by a power of two
                    const int up = min(137 - static_cast<int>(__float_as_uint(top) >> 23), 120);
                    const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                    if (c == 0)
                        cq_of[(KS ? 0 : 128 * g) + rk] = fmaxf(A.scale * kLog2e * (FMT == kKv8 ? 0.0625f : 1.0f) *
                                                               __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 1.2e-38f);
#pragma unroll
                    for (int u = 0; u < 8; ++u) f[u] *= by;
                    *reinterpret_cast<uint4 *>(sm + (KS ? 0 : g * Q::Q_BYTES) + rk * 128 + (c >> 3) * (128 * 128) + (((c & 7) ^ (rk & 7)) << 4)) =
                        make_uint4(pack_h(f[0], f[4]), pack_h(f[1], f[5]), pack_h(f[2], f[6]), pack_h(f[3], f[7]));
                }
            }
            if (!KS || g == 0) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();            // group 0 has read both accumulators of the segment before
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kQFull));
            } else if (!__all_sync(0xffffffffu, wait(kQFull, seg_no))) {         // group 0 has taken the state of the segment before
                return false;
            }
            const float cq = cq_of[(KS ? 0 : 128 * g) + r], slope2 = X && A.slopes ? A.slopes[hq] * kLog2e : 0.0f;
            const int all_hi = tree.base, all_lo = first_seen(A, use.s.hi - 1);
            float mref = -INFINITY, mz = 0.0f, lsum = 0.0f;
#pragma unroll 1
            for (int k = KS ? g : 0, buf = (i0 + k) % Q::BUFS, row0 = use.s.lo + (run.f0 + i0 + k - use.base) * SR; k < n;
                 k += STRIDE, ++cnt, row0 += STRIDE * SR, buf = buf + STRIDE >= Q::BUFS ? buf + STRIDE - Q::BUFS : buf + STRIDE) {
                const int b = cnt & 1;
                const bool begins = k < STRIDE, masked = row0 < all_lo || row0 + SR > all_hi;
                const uint32_t tS = tq + 64 * (2 * g + b);
                if (!__all_sync(0xffffffffu, wait(kSFull + 2 * g + b, cnt >> 1))) return false;
                if (active) {
                    tc_fence_after();
                    uint32_t s[64];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc_ld16(tS + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(s + 16 * c));
                    tc_wait_ld();
                    const float *f = reinterpret_cast<const float *>(scales + buf * Q::SCALES);
                    const int2 info = about[buf];
                    const uint32_t gone = info.x;
                    const int E = info.y;
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
                    uint32_t vis[2] = {0xffffffffu, 0xffffffffu};
                    if (masked || gone) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            vis[h] = masked ? seen32(tree, m, from, row0 + 32 * h) : 0xffffffffu;
                            if (gone >> (2 * h) & 1u) vis[h] &= 0xffff0000u;
                            if (gone >> (2 * h + 1) & 1u) vis[h] &= 0x0000ffffu;
                        }
                    }
                    if constexpr (X) {
                        if (A.softcap > 0.0f) {
                            if (masked || gone) {
#pragma unroll
                                for (int j = 0; j < 64; ++j) s[j] = vis[j >> 5] >> (j & 31) & 1u ? s[j] : 0u;
                            }
                            cap_all(reinterpret_cast<float(&)[64]>(s), cap2, inv2);
                        }
                        if (A.slopes) {
                            if (row0 + SR > tree.base) {
#pragma unroll
                                for (int j = 0; j < 64; ++j)
                                    s[j] = __float_as_uint(fmaf(slope2, static_cast<float>(tree.position(row0 + j) - own), __uint_as_float(s[j])));
                            } else {
#pragma unroll
                                for (int j = 0; j < 64; ++j) s[j] = __float_as_uint(fmaf(slope2, static_cast<float>(row0 + j - own), __uint_as_float(s[j])));
                            }
                        }
                    }
                    if (masked || gone) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) s[j] = vis[j >> 5] >> (j & 31) & 1u ? s[j] : 0xFF800000u;
                    }
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, top;
                    if (E != kCodes) {        // the largest score, and V's power of two
#pragma unroll
                        for (int j = 0; j < 64; ++j) tops[j & 3] = fmaxf(tops[j & 3], __uint_as_float(s[j]));
                        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                        top = X ? top + static_cast<float>(E) : fmaf(top, cq, static_cast<float>(E));
                    } else {                  // scores with the log2 of V's scales
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
                        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    }
                    if (__any_sync(0xffffffffu, top > mref + slack<FMT>())) {
                        const float mn = top > mref + slack<FMT>() ? top - lead<FMT>() : mref, alpha = ex2(mref == -INFINITY ? -INFINITY : mref - mn);
                        mref = mn;
                        mz = mn == -INFINITY ? 0.0f : mn;
                        lsum *= alpha;
                        if (!begins) {        // O of the steps before, once their product is complete
                            if (!__all_sync(0xffffffffu, wait(kPvDone + 2 * g + (b ^ 1), (cnt - 1) >> 1))) return false;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tc_ld16(to + 16 * c, o);
                                tc_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tc_st16(to + 16 * c, o);
                            }
                            tc_wait_st();
                        }
                    }
                    unsigned long long sum0 = zero2, sum1 = zero2;
                    const float less1 = E == kCodes ? -mz : static_cast<float>(E) - mz;
                    const unsigned long long less = f2_pack(less1, less1);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pr[16];
                        auto exps = [&](int q, unsigned long long &e0, unsigned long long &e1) {
                            const unsigned long long x0 = f2_pack(__uint_as_float(s[q]), __uint_as_float(s[q + 1])),
                                                     x1 = f2_pack(__uint_as_float(s[q + 2]), __uint_as_float(s[q + 3]));
                            const float2 a0 = f2_unpack(X ? f2_add(x0, less) : f2_fma(x0, cq2, less)),
                                         a1 = f2_unpack(X ? f2_add(x1, less) : f2_fma(x1, cq2, less));
                            e0 = f2_pack(ex2(a0.x), ex2(a0.y));
                            e1 = f2_pack(ex2(a1.x), ex2(a1.y));
                            sum0 = f2_add(sum0, e0);
                            sum1 = f2_add(sum1, e1);
                        };
                        if (E != kCodes) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                unsigned long long e0, e1;
                                exps(32 * c + j, e0, e1);
                                const float2 p0 = f2_unpack(e0), p1 = f2_unpack(e1);
                                pr[j / 2] = pack_h(p0.x, p0.y);
                                pr[j / 2 + 1] = pack_h(p1.x, p1.y);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 v4 = *reinterpret_cast<const float4 *>(f + kKeys + 32 * c + j);
                                unsigned long long e0, e1;
                                exps(32 * c + j, e0, e1);
                                const float2 p0 = f2_unpack(f2_fma(e0, f2_pack(v4.x, v4.y), zero2)), p1 = f2_unpack(f2_fma(e1, f2_pack(v4.z, v4.w), zero2));
                                pr[j / 2] = pack_h(p0.x, p0.y);
                                pr[j / 2 + 1] = pack_h(p1.x, p1.y);
                            }
                        }
                        tc_st16(tS + 16 * c, pr);
                    }
                    // of the weights without V's power of two
                    const float2 sum = f2_unpack(f2_add(sum0, sum1));
                    lsum = fmaf(sum.x + sum.y, __uint_as_float(static_cast<uint32_t>(127 - (E == kCodes ? 0 : E)) << 23), lsum);
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + 2 * g + b));
            }

            // ---- the segment's end: the group's last product
            if (n > (KS ? g : 0) && !__all_sync(0xffffffffu, wait(kPvDone + 2 * g + (cnt - 1 & 1), (cnt - 1) >> 1))) return false;
            if (KS && g == 1) {
                state[r] = make_float2(mref, lsum);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kState));
                return true;
            }
            float f0 = 1.0f, f1 = 0.0f;
            if constexpr (KS) {
                if (!__all_sync(0xffffffffu, wait(kState, seg_no))) return false;
                const float2 two = state[r];
                const float mn = fmaxf(mref, two.x), mm = mn == -INFINITY ? 0.0f : mn;
                f0 = ex2(mref - mm);
                f1 = ex2(two.x - mm);
                mref = mn;
                lsum = lsum * f0 + (n > 1 ? two.y * f1 : 0.0f);
            }
            const bool starts = use.base >= run.f0, ends = use.base + use.s.steps <= run.f1, whole = starts && ends;
            if (active) {
                tc_fence_after();
                if (!used) {                  // its query may have been anything
                    mref = -INFINITY;
                    lsum = 0.0f;
                }
                const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (starts ? 1 : 0)) * A.cols;
                const float fo = (FMT == kKv8 ? 0.0625f : 1.0f) * (!whole ? 1.0f : lsum == 0.0f ? 0.0f : 1.0f / lsum);
                f0 *= fo;
                f1 *= fo;
                if (!whole && valid) *reinterpret_cast<float2 *>(A.part_ml + 2 * (slot + row)) = make_float2(mref, lsum);
                // a thread has a row, but 32 rows are written 128 bytes at a time: they turn in the warp's share of Q's
                // place, which no product reads any more
                unsigned char *turn = sm + (KS ? 0 : g * Q::Q_BYTES) + (r & ~31) * 128;
                auto columns = [&](int c, float (&x)[16]) {      // of the row, in the order of the dimensions
                    uint32_t o[16];
                    tc_ld16(to + c, o);
                    tc_wait_ld();
                    // columns 0 4 1 5 2 6 3 7 of each eight dimensions
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[(e & 8) + ((e & 7) >> 1) + 4 * (e & 1)] = used ? __uint_as_float(o[e]) * f0 : 0.0f;
                    if (KS && n > 1) {        // (of one step group 1 has had none, and its accumulator may hold anything)
                        tc_ld16(to + 128 + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int d = (e & 8) + ((e & 7) >> 1) + 4 * (e & 1);
                            x[d] = used ? fmaf(__uint_as_float(o[e]), f1, x[d]) : 0.0f;
                        }
                    }
                };
                auto put = [&](int k, uint4 v) { *reinterpret_cast<uint4 *>(turn + lane * 128 + ((k ^ (lane & 7)) << 4)) = v; };
                auto rows_out = [&](auto address) {              // address(row of the tile, its 16-byte chunk)
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int rr = 4 * k + lane / 8, vk = (row & ~31) + rr;
                        if (vk < nv) *reinterpret_cast<uint4 *>(address(vk, lane & 7)) = *reinterpret_cast<const uint4 *>(turn + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                    }
                    __syncwarp();
                };
                if (whole) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 64) {
#pragma unroll 1
                        for (int h = 0; h < 4; ++h) {
                            float x[16];
                            columns(c + 16 * h, x);
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                put(2 * h + k, make_uint4(pack_b(x[8 * k], x[8 * k + 1]), pack_b(x[8 * k + 2], x[8 * k + 3]),
                                                          pack_b(x[8 * k + 4], x[8 * k + 5]), pack_b(x[8 * k + 6], x[8 * k + 7])));
                        }
                        rows_out([&](int vk, int k) {
                            const int mk = row_of_vector(A, v0 + vk);
                            return A.out + ((static_cast<size_t>(use.b) * A.M + mk) * A.Hq + kvh * A.G + v0 + vk - mk * A.G) * D + c + 8 * k;
                        });
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            float x[16];
                            columns(c + 16 * h, x);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                put(4 * h + k, make_uint4(__float_as_uint(x[4 * k]), __float_as_uint(x[4 * k + 1]), __float_as_uint(x[4 * k + 2]), __float_as_uint(x[4 * k + 3])));
                        }
                        rows_out([&](int vk, int k) { return A.part_o + (slot + vk) * D + c + 4 * k; });
                    }
                }
            }
            if (i0 + n == steps && threadIdx.x == 0 && !ends && starts)
                A.info[blockIdx.x] = make_int4(use.b, use.seg, (use.base + use.s.steps - 1 + (run.seg + seg_no + 1) * kSegCost) / run.per, 0);
            return true;
        };
#pragma unroll 1
        while (segment()) {
            i0 += use.end - max(use.base, run.f0);
            ++seg_no;
            if (i0 >= steps) break;
            use.next(A, segs);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && abort_flag) A.info[blockIdx.x] = make_int4(-1, 0, 0, 0);   // some of what would be joined may be missing
    if (warp == kMmaWarp && keep_tmem == 0) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

template <int FMT, int D, bool X, bool KS>
cudaError_t launch(const AttnArgs &A, cudaStream_t s, int *grid)
{
    using Q = Tt<FMT, D, KS>;
    static std::atomic<bool> done[64];          // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev].load()) {
        e = cudaFuncSetAttribute(attn_tree_tc_kernel<FMT, D, X, KS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q::SMEM);
        if (e != cudaSuccess) return e;
        done[dev].store(true);
    }
    *grid = sm_count();
    attn_tree_tc_kernel<FMT, D, X, KS><<<*grid, kThreads, Q::SMEM, s>>>(A);
    return cudaGetLastError();
}
template <int FMT, int D>
cudaError_t launch_x(const AttnArgs &A, cudaStream_t s, int *grid)
{
    const bool x = A.softcap > 0.0f || A.slopes;
    if (A.cols <= 128) return x ? launch<FMT, D, true, true>(A, s, grid) : launch<FMT, D, false, true>(A, s, grid);
    return x ? launch<FMT, D, true, false>(A, s, grid) : launch<FMT, D, false, false>(A, s, grid);
}

}  // namespace

cudaError_t attn_tree_tc(int fmt, const AttnArgs &A, cudaStream_t s, int *grid)
{
    if (fmt == kKv4) return A.p.D == 128 ? launch_x<kKv4, 128>(A, s, grid) : launch_x<kKv4, 64>(A, s, grid);
    return A.p.D == 128 ? launch_x<kKv8, 128>(A, s, grid) : launch_x<kKv8, 64>(A, s, grid);
}

}  // namespace nq
