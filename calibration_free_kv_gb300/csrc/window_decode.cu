// Windowed decode: the persistent decode kernels over the pages a sliding window and the first
// tokens leave visible (decode_kernel.cuh with WIN).  A query reads ceil(sink / 128) + window / 128
// pages and their edges whatever the sequence's length: the pages in between are never looked up.
#include "common.cuh"
#include "decode_kernel.cuh"
#include "params.cuh"

namespace kvarn {

int launch_window_decode(int d, int nt, int kb, int vb, const DecodeParams& p, cudaStream_t stream) {
  const int phases = kDecodeSplits | kDecodeMerge;
  if (kb == 4 && vb == 2) return launch_decode_bits<4, 2, true>(d, nt, p, phases, stream);
  if (kb == 4 && vb == 4) return launch_decode_bits<4, 4, true>(d, nt, p, phases, stream);
  if (kb == 2 && vb == 2) return launch_decode_bits<2, 2, true>(d, nt, p, phases, stream);
  if (kb == 8 && vb == 4) return launch_decode_bits<8, 4, true>(d, nt, p, phases, stream);
  return KVARN_ERR_UNSUPPORTED;
}

}  // namespace kvarn
