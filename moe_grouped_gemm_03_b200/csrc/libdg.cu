// The library's one translation unit: the grouped GEMMs (dg_api.cu) and the operators around them (moe_ops.cuh).
#include "dg_api.cu"
#include "moe_ops.cuh"
