// Attention within each molecule on tensor cores, bf16 storage: the key side of the backward pass.
#include "molecule_bwd_k_tc.cuh"

namespace egat {

int mol_tc_backward_k_bf16(const MolParams& p, cudaStream_t st) { return tc_backward_k<1>(p, st); }

}  // namespace egat
