// pt_decode_tc.cu -- tensor-core kernels of the decoding attention (bf16).
#include "pt.h"
#include "pt_decode.cuh"
#include "pt_internal.h"

namespace pt {

int take_status_decode_tc(cudaStream_t s) { return take_status_here(s); }

bool decode_tc_supported(int D, int ps) { return false; }

int decode_tc(const pt_decodeplan* p, DecArgs a, DecClass rows, DecClass tile, cudaStream_t s) { return PT_ERR_UNSUPPORTED; }

}  // namespace pt
