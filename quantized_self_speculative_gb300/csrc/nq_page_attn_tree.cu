// nq_page_attn_tree.cu -- attention of trees over pages, up to 16 query vectors per kv
// head: the T form of nq_page_attn_warp.cuh.
//
// Node m of a tree of M nodes lies in row base + m.  The committed rows are seen by
// every node and need no mask; only the steps that reach the tree's rows (and those
// at a window's border) test a bit per score.  All trees take the form for capped or
// biased scores, whatever theirs are, and join_tree_kernel joins their parts.
// Measured (GB300): a tree of 16 nodes over 533 rows, 32 kv heads of 128, 8-bit view:
// 20 us, bound by the latency of one short run and the join.  us of trees / of causal rows,
// 8 kv heads of 128, 8-bit view, 8 and 16 vectors: 16 sequences of 500..4000 rows 28.8 / 26.9
// and 41.1 / 36.9 (27.0 and 37.5 with a form without caps); one of 32768 rows 34.9 / 24.6
// and 43.1 / 30.8, where segments have some 50 parts (26.8 and 36.8 with the causal join).
#include "nq_page_attn_warp.cuh"

namespace nq {

cudaError_t attn_tree(int fmt, const AttnArgs &A, cudaStream_t s, int *grid)
{
    const int nt = A.cols / 8;
    return fmt == kBf16 ? launch_d<kBf16, true>(nt, A, s, grid) : fmt == kKv4 ? launch_d<kKv4, true>(nt, A, s, grid) : launch_d<kKv8, true>(nt, A, s, grid);
}

}  // namespace nq
