// flexq_lib.cu -- the library's one translation unit: the 6-bit path and the
// 4-bit / table operators share the error message, the argument checks and
// the device status word of flexq_api.cu without relocatable device code.
#include "flexq_api.cu"
#include "flexq_w4_api.cuh"
