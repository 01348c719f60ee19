// nq_page_attn_tree.cu -- attention of trees over pages, up to 16 query vectors per kv
// head: the T form of nq_page_attn_warp.cuh.
//
// Node m of a tree of M nodes lies in row base + m.  The committed rows are seen by
// every node and need no mask; only the steps that reach the tree's rows (and those
// at a window's border) test a bit per score.  A step over the prefix costs what
// it costs without trees.  Measured (GB300): a tree of 16 nodes over 533 rows, 32 kv heads
// of 128, 8-bit view: 20 us, bound by the latency of one short run and the join.
#include "nq_page_attn_warp.cuh"

namespace nq {

cudaError_t attn_tree(int fmt, const AttnArgs &A, cudaStream_t s, int *grid)
{
    const int nt = A.cols / 8;
    return fmt == kBf16 ? launch_d<kBf16, true>(nt, A, s, grid) : fmt == kKv4 ? launch_d<kKv4, true>(nt, A, s, grid) : launch_d<kKv8, true>(nt, A, s, grid);
}

}  // namespace nq
