// The INT4 cache tile and its group quantiser, shared by the kernels that
// write, read and move the cache.
#pragma once

#include <math_constants.h>

#include "kvq_common.cuh"

namespace kvq {

// INT4 tile of one (page, KV head): see kvq_int4_tile_bytes in kvq.h.
constexpr int INT4_TILE = 2560;
constexpr int O4_KC = 0, O4_KM = 1024, O4_VC = 1280, O4_VS = 2304, O4_VM = 2432;
constexpr int INT4_LEVELS = 15;  // highest code

__host__ __device__ constexpr int int4_vmeta_off(int s, int g) { return 16 * (s >> 1) + 4 * g + 2 * (s & 1); }

// fp32 -> fp16 round-to-nearest-even, saturating at +-65504; NaN stays NaN.
__device__ __forceinline__ __half f16_sat_nan(float x) { return x != x ? __float2half_rn(x) : f16_sat(x); }

// Group parameters and codes from the exact rotated values: the range ends
// and their difference are taken in fp64, and each parameter is rounded to
// fp32 and then to fp16, as the format states.
__device__ __forceinline__ void int4_params(double mn, double mx, double clip, __half& sh, __half& mh) {
    mn *= clip;
    mx *= clip;
    sh = f16_sat_nan(__double2float_rn((mx - mn) / (double)INT4_LEVELS));
    mh = f16_sat_nan(__double2float_rn(mn));
}

// #{c in 0..14 : min + (c + 1/2) scale < z}.  The quotient of an exact tie is
// exactly c + 1/2, so ties go to the lower level.
__device__ __forceinline__ int int4_code(double z, __half sh, __half mh) {
    const double sc = (double)__half2float(sh);
    if (!(sc > 0.0)) return 0;
    const double c = ceil((z - (double)__half2float(mh)) / sc - 0.5);
    return c > 0.0 ? (c < (double)INT4_LEVELS ? (int)c : INT4_LEVELS) : 0;
}

}  // namespace kvq
