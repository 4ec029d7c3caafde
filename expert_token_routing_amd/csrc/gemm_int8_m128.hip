// The int8 grouped GEMMs with 128-row tiles and a third ring slot, for batches
// in which each expert sees few rows (the decode regime), as the bf16 ones in
// gemm_bf16_m128.hip: such launches stream the weights from HBM.
#define OCC_GEMM_TILE_M 128
#define OCC_GEMM_NSTAGE 3
#define OCC_GEMM_SUFFIX _m128
#include "gemm_int8.hip"
