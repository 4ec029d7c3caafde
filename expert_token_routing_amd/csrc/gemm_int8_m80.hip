// The int8 grouped GEMMs for batches in which each expert sees few rows (the
// decode regime).  Such launches stream the weights from HBM, so what counts
// is how many bytes are in flight on a CU at any time: 80 x 128 tiles (64
// features of the up-projection) in a ring of three, two workgroups on a CU,
// whose starts and ends fall beside the other's stream.  Measured on the layer
// (d = 2048, 64 experts of F = 1024, top 8, an uneven router) against 128 x 256
// tiles, one workgroup on a CU: T = 16 / 128 / 256 / 512 / 767 69 / 97 / 110 /
// 128 / 151 us against 74 / 102 / 120 / 137 / 150; 64-row tiles are even below
// 64 rows an expert and slower above (132 us at T = 512), 240-row tiles 6 to
// 12% slower throughout.  320-row tiles overtake at some 128 rows an expert (182 against
// 178 us at T = 1023).  Streaming the weights into registers past LDS lost (207
// us at T = 512): there the rows of codes have to be read by every wave.
#define OCC_GEMM_TILE_M 80
#define OCC_GEMM_TILE_N 128
#define OCC_GEMM_WG_PER_CU 2
#define OCC_GEMM_NSTAGE 3
#define OCC_GEMM_SUFFIX _m80
#include "gemm_int8.hip"
