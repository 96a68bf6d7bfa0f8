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

// The parameters from fp32 ends known to within eps (in absolute terms), and
// whether the exact ends could give others: bit 0 another min, bit 1 another scale.
// Rounding to fp32 and then to fp16 is monotone, so they are certain when both ends
// of their intervals round alike (what saturates counts as open).
__device__ __forceinline__ int int4_params_near(float mn, float mx, float clip, float eps, __half& sh, __half& mh) {
    const float s = clip * (mx - mn) * (1.f / INT4_LEVELS), m = clip * mn;
    const float ds = fmaf(clip * (2.f / INT4_LEVELS), eps, s * 0x1p-21f), dm = fmaf(clip, eps, fabsf(m) * 0x1p-22f);
    const __half2 lo = __floats2half2_rn(s - ds, m - dm), hi = __floats2half2_rn(s + ds, m + dm);
    sh = __low2half(lo);
    mh = __high2half(lo);
    const uint32_t diff = h2_as_u32(lo) ^ h2_as_u32(hi);
    return (diff >> 16 != 0 || !(fabsf(m) + dm < 65504.f)) | ((diff & 0xffff) != 0 || !(s + ds < 65504.f)) << 1;
}

// Unevaluated sums hi + lo of two fp32 values (about 46 bits).
struct Dd {
    float hi, lo;
};

// acc + (x + xl) r
__device__ __forceinline__ void dd_fma(Dd& acc, float x, float xl, float r) {
    const float p = __fmul_rn(x, r), e = __fmaf_rn(xl, r, __fmaf_rn(x, r, -p));
    float s, t;
    two_sum(acc.hi, p, s, t);
    acc.hi = s;
    acc.lo = __fadd_rn(acc.lo, __fadd_rn(t, e));
}

__device__ __forceinline__ void dd_add(Dd& acc, Dd o) {
    float s, t;
    two_sum(acc.hi, o.hi, s, t);
    acc.hi = s;
    acc.lo = __fadd_rn(acc.lo, __fadd_rn(t, o.lo));
}

// hi the nearest fp32 to the sum, so that pairs compare by hi, then lo
__device__ __forceinline__ Dd dd_norm(Dd a) {
    Dd r;
    two_sum(a.hi, a.lo, r.hi, r.lo);
    return r;
}
__device__ __forceinline__ bool dd_less(Dd a, Dd b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }

// The parameters from exact ends in pairs: the quotient by 15 is refined by its
// exact remainder, and the sum of the two parts is one rounding to fp32.
__device__ __forceinline__ void int4_params(Dd mn, Dd mx, float clip, __half& sh, __half& mh) {
    Dd d = {mx.hi, mx.lo};
    dd_add(d, Dd{-mn.hi, -mn.lo});
    d = dd_norm(d);
    float p = __fmul_rn(clip, d.hi), e = __fmaf_rn(clip, d.lo, __fmaf_rn(clip, d.hi, -p));
    const float q = __fdiv_rn(p, (float)INT4_LEVELS), rest = __fadd_rn(__fmaf_rn(-q, (float)INT4_LEVELS, p), e);
    sh = f16_sat_nan(__fadd_rn(q, __fdiv_rn(rest, (float)INT4_LEVELS)));
    p = __fmul_rn(clip, mn.hi);
    e = __fmaf_rn(clip, mn.lo, __fmaf_rn(clip, mn.hi, -p));
    mh = f16_sat_nan(__fadd_rn(p, e));
}

// code of z near threshold n (code n or n + 1): min + (n + 1/2) scale is a sum of
// two fp32 values exactly, and z minus it has the right sign.
__device__ __forceinline__ int int4_code(Dd z, float s, float m, int n) {
    float th, tl, d, e;
    two_sum(m, ((float)n + 0.5f) * s, th, tl);
    two_sum(z.hi, -th, d, e);
    return n + (__fadd_rn(d, __fadd_rn(e, __fsub_rn(z.lo, tl))) > 0.f);
}

// Sums of squares outside this range (and not 0) leave the fp32 paths: products
// would lose bits below the smallest fp32 or leave its range.
__device__ __forceinline__ bool int4_wild(float n2) { return !(n2 == 0.f || (n2 > 0x1p-80f && n2 < 0x1p100f)); }

}  // namespace kvq
