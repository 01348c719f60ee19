// nq_page_attn_wide.cu -- attention over pages for more than 16 query vectors
// per kv head (a verify pass with grouped queries: k + 1 rows times the group):
// nested pages up to 24 (heads of 64: 32), and beyond where the tensor-core kernel
// does not serve (bf16 pages, two scales per row).
//
// The same list of steps and the same arithmetic as nq_page_attn.cu, but here
// decoding the codes and the products bound the time, not HBM: with 20 query
// vectors that kernel would decode every block for each of two tiles.  So a CTA
// decodes a step once, into fp16 tiles in shared memory (codes as signed
// numbers, exact; the scales stay apart), and its four or eight warps hold the
// query columns between them, a tile of 8 each: every warp takes all rows for its
// own columns, and nothing is merged within a CTA.  While the warps work on
// one step they decode the next; one barrier per step.  bf16 pages need no
// decoding: the ring's stages are the tiles.
// Measured (GB300): 16 sequences of 500..4000 rows, 8 kv heads of 128, 20 query
// vectors each, 8-bit view: 59 us for 90 MB, bound by the latency between its
// barriers (decode, S, softmax, O), not by HBM (13 us) or the MMA pipe.  bf16 pages:
// 63 us for 176 MB, with 36 vectors 81; two scales per row, 36 vectors: 92 us.
#include "nq_page_attn_wide.cuh"

namespace nq {

cudaError_t attn_wide(int fmt, const AttnArgs &A, cudaStream_t s, int *grid)
{
    const int warps = A.cols / 8;
    return fmt == kBf16 ? launch_d<kBf16, false>(A, warps, s, grid) : fmt == kKv4 ? launch_d<kKv4, false>(A, warps, s, grid) : launch_d<kKv8, false>(A, warps, s, grid);
}

}  // namespace nq
