// Attention within each molecule on tensor cores, float32 storage: the key side of the backward pass.
#include "molecule_bwd_k_tc.cuh"

namespace egat {

int mol_tc_backward_k_f32(const MolParams& p, cudaStream_t st) { return tc_backward_k<3>(p, st); }

}  // namespace egat
