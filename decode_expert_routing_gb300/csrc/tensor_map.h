// cuTensorMapEncodeTiled, from the driver through the runtime's entry-point
// query (the library links only the CUDA runtime).
#pragma once

#include <cuda.h>

namespace mr {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled();  // nullptr when the driver has no such entry point

}  // namespace mr
