// Attention within each molecule on tensor cores, float32 storage: the forward pass.
#include "molecule_fwd_tc.cuh"

namespace egat {

int mol_tc_forward_f32(const MolParams& p, cudaStream_t st) { return tc_forward<3>(p, st); }

}  // namespace egat
