// dq_tma_host.h -- the driver's tensor-map encoder, looked up once per process.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace dqhost {

using EncodeTiled = PFN_cuTensorMapEncodeTiled_v12000;

EncodeTiled encode_tiled();  // null where the driver has none

}  // namespace dqhost
