// Rows of packed sequences: their positions, and zeros in rows of nobody.
#include "varlen.cuh"

namespace tpmlp {
namespace {

// A warp a row.  Bound by the stores; the search over cu_rows is one to four
// probes of 32 entries.
__global__ void __launch_bounds__(256) packed_rows_kernel(const SeqRows s, int32_t* pos, uint4* z, int64_t z16,
                                                          uint4* dz, int64_t dz16) {
  const int lane = threadIdx.x & 31;
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < s.rows; row += (int64_t)gridDim.x * 8) {
    const int b = find_row(s, (int)row, lane);
    bool bad = false;  // reported by the attention kernels
    const SeqSpan sp = seq_span(s, b, -1, &bad);
    const bool mine = row >= sp.first && row - sp.first < sp.count;
    if (pos && lane == 0) pos[row] = mine ? (int)row - sp.first : 0;
    if (mine) continue;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t i = lane; z && i < z16; i += 32) z[row * z16 + i] = zero;
    for (int64_t i = lane; dz && i < dz16; i += 32) dz[row * dz16 + i] = zero;
  }
}

}  // namespace

cudaError_t launch_packed_rows(const SeqRows& s, int32_t* pos, void* z, int64_t z_bytes, void* dz, int64_t dz_bytes,
                               int num_sms, cudaStream_t st) {
  const int64_t want = (s.rows + 7) / 8, most = 8LL * num_sms;
  packed_rows_kernel<<<(unsigned)(want < most ? want : most), 256, 0, st>>>(s, pos, static_cast<uint4*>(z), z_bytes / 16,
                                                                            static_cast<uint4*>(dz), dz_bytes / 16);
  return cudaGetLastError();
}

}  // namespace tpmlp
