// q8_gemm.hip -- launches of the 8-bit products with one scale per token and
// one per output channel, dense and over experts (kernels: q8_kernels.hpp).
#include "q8_kernels.hpp"

namespace coli {

static Variant variant_of(const Q8Args &a) { return a.offs ? grouped_variant(a) : dense_variant(a); }

bool gemm_q8_fits(const Q8Args &a) {
  // (the grouped kernels name rows of q by 32-bit byte offsets)
  if (a.offs && (int64_t)a.rows * a.K >= (int64_t)1 << 32) return false;
  const Variant v = variant_of(a);
  return workgroups(a, v) * kShapes[v].threads < ((int64_t)1 << 31);
}

hipError_t launch_gemm_q8(int dt, const Q8Args &a, hipStream_t st) {
  if ((a.offs ? a.P : a.rows) == 0) return hipSuccess;
  const Variant v = variant_of(a);
  const int64_t wgs = workgroups(a, v);
  return by_dtype(dt, [&](auto dtc) {
    constexpr int DT = decltype(dtc)::value;
    if (!a.offs) {
      run_dense<DT>(a, v, st);
    } else {
      switch (v) {
        case kRing16x32: run_ring<DT, true, 16, 32, 1, 1, 4, 3>(a, wgs, st); break;
        case kRing64x32: run_ring<DT, true, 64, 32, 2, 1, 4, 3>(a, wgs, st); break;
        case kSweep32: run_sweep<DT, true, 32, 2, 4>(a, wgs, st); break;
        case kSweep64: run_sweep<DT, true, 64, 4, 3>(a, wgs, st); break;
        default: run_tile<DT, true, 256, 256, 1, 8, 157 << 10>(a, wgs, st); break;
      }
    }
    return hipGetLastError();
  });
}

}  // namespace coli
