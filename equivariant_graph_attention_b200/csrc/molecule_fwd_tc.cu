// Attention within each molecule on tensor cores, bf16 storage: the forward pass.
#include "molecule_fwd_tc.cuh"

namespace egat {

int mol_tc_forward_bf16(const MolParams& p, cudaStream_t st) { return tc_forward<1>(p, st); }

}  // namespace egat
