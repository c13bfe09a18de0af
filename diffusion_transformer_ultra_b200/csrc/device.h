// The device a call runs on, and the driver's tensor map encoder (api.cu).
#pragma once

#include <cuda.h>

namespace ug {

// The current device, or ULTRAGEN_ERR_NO_DEVICE when it is not an sm_100 one.
int current_device(int* dev);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled, or null when the driver has none.
EncodeTiledFn encode_fn();

}  // namespace ug
