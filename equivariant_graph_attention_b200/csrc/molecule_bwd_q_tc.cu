// Attention within each molecule on tensor cores, bf16 storage: the query side of the backward pass.
#include "molecule_bwd_q_tc.cuh"

namespace egat {

int mol_tc_backward_q_bf16(const MolParams& p, cudaStream_t st) { return tc_backward_q<1>(p, st); }

}  // namespace egat
