// Attention within each molecule on tensor cores, float32 storage: the query side of the backward pass.
#include "molecule_bwd_q_tc.cuh"

namespace egat {

int mol_tc_backward_q_f32(const MolParams& p, cudaStream_t st) { return tc_backward_q<3>(p, st); }

}  // namespace egat
