// nq_page_attn_tree_wide.cu -- attention of trees over pages for more than 16 query
// vectors per kv head where the tensor-core kernel does not serve (bf16 pages, two
// scales per row): the T form of nq_page_attn_wide.cuh (masks as in nq_page_attn_tree.cu).
// Measured (GB300): 8 sequences of 900..9001 rows, 4 kv heads of 64, bf16, trees of up to 13
// nodes, 52 vectors under a cap, a bias and a window of 4096: 35 us for 26 MB.  16
// sequences of 500..4000 rows, 8 kv heads of 128, 36 / 128 / 256 vectors: bf16 75 / 174 /
// 353 us, two scales per row (8-bit view) 88 / 192 / 369.  Bound by the latency between
// its barriers, once per tile of 64 vectors: each tile reads and decodes the rows again.
#include "nq_page_attn_wide.cuh"

namespace nq {

cudaError_t attn_tree_wide(int fmt, const AttnArgs &A, cudaStream_t s, int *grid)
{
    const int warps = A.cols / 8;
    return fmt == kBf16 ? launch_d<kBf16, true>(A, warps, s, grid) : fmt == kKv4 ? launch_d<kKv4, true>(A, warps, s, grid) : launch_d<kKv8, true>(A, warps, s, grid);
}

}  // namespace nq
