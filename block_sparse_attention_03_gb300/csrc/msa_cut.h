// How a batch with more units than one launch of the dense attend counts (32 bits) is cut.  No CUDA here: the host
// tests compile it by itself.
#pragma once

namespace msa {

// Sequences [s0, s0 + n) of a call, and where their parts of its arrays begin, in elements.
struct DenseCut {
  long s0, n;
  long table;  // block_table [seqs][max_nb]
  long lists;  // topk_idx [seqs][tokens][G][topk]
  long row;    // rows of q, out and lse: [seqs][tokens][hq]
};

// units: of a sequence; limit: of a launch, no less than that.
inline DenseCut dense_cut(long s0, long seqs, long units, long limit, long tokens, int hq, int max_nb, int G, int topk) {
  const long most = limit / units;
  DenseCut c;
  c.s0 = s0;
  c.n = seqs - s0 < most ? seqs - s0 : most;
  c.table = s0 * max_nb;
  c.lists = s0 * tokens * G * topk;
  c.row = s0 * tokens * hq;
  return c;
}

}  // namespace msa
