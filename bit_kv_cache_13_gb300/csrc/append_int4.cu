// Quantise-on-append and read-back of the rotated INT4 KV cache.
//
// z = (k - mu) R_k, w = v R_v, then 16 levels per group of 32 rotated channels
// with an fp16 scale and min.  Codes, scales and mins are those of the exact
// rotated vectors, whichever kernel writes them.
#include "int4_common.cuh"

namespace kvq {

// One CTA of 256 threads per (token, KV head): thread j < 128 forms rotated
// key channel j, thread 128 + j value channel j, as fp64 dot products of the
// exact inputs (k - mu of a bf16 and an fp32 is exact in fp64).  Warp w is
// group w % 4 of side w / 4, so a group's range is a warp reduction.
__global__ void __launch_bounds__(256)
append_int4_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v, int n_tok, int H_kv,
                   const int32_t* __restrict__ slot_mapping, const float* __restrict__ mu,
                   const float* __restrict__ Rk, const float* __restrict__ Rv, uint8_t* __restrict__ cache,
                   int64_t num_pages, int32_t* __restrict__ err_count, float clip) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ double xs[2][D];
    const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int side = tid >> 7, j = tid & (D - 1), lane = tid & 31, g = (tid >> 5) & 3;
    const int slot = __ldg(slot_mapping + t);
    if (slot == -1) return;
    if (slot < 0 || (int64_t)slot >= num_pages * PAGE) {
        if (tid == 0 && h == 0 && err_count) atomicAdd(err_count, 1);
        return;
    }
    const size_t row = ((size_t)t * H_kv + h) * D + j;
    xs[side][j] = side ? (double)__bfloat162float(v[row])
                       : (double)__bfloat162float(k[row]) - (double)__ldg(mu + (size_t)h * D + j);
    __syncthreads();
    const float* R = (side ? Rv : Rk) + (size_t)h * D * D + j;
    double z = 0.0;
#pragma unroll 8
    for (int i = 0; i < D; ++i) z = fma(xs[side][i], (double)__ldg(R + (size_t)i * D), z);
    double mn = z, mx = z;
    const bool nan = !isfinite(z);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        mn = fmin(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if (__any_sync(0xffffffffu, nan)) mn = mx = CUDART_NAN;
    __half sh, mh;
    int4_params(mn, mx, (double)clip, sh, mh);
    const int code = int4_code(z, sh, mh);
    uint8_t* tile = cache + ((size_t)(slot / PAGE) * H_kv + h) * INT4_TILE;
    const int s = slot % PAGE;
    if (!side) {
        // word (t = lane / 8, g): nibble lane % 8
        uint32_t w = (uint32_t)code << (4 * (lane & 7));
        w |= __shfl_xor_sync(0xffffffffu, w, 1);
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
        w |= __shfl_xor_sync(0xffffffffu, w, 4);
        if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(tile + O4_KC + 64 * s + 16 * (lane >> 3) + 4 * g) = w;
        if (lane == 0) {
            *reinterpret_cast<__half*>(tile + O4_KM + 16 * s + 2 * g) = sh;
            *reinterpret_cast<__half*>(tile + O4_KM + 16 * s + 8 + 2 * g) = mh;
        }
    } else {
        // half s % 2 of the word (r = lane / 4, g) of slot pair s / 2: nibble lane % 4
        uint32_t w = (uint32_t)code << (4 * (lane & 3));
        w |= __shfl_xor_sync(0xffffffffu, w, 1);
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
        if ((lane & 3) == 0)
            *reinterpret_cast<uint16_t*>(tile + O4_VC + 128 * (s >> 1) + 16 * (lane >> 2) + 4 * g + 2 * (s & 1)) =
                (uint16_t)w;
        if (lane == 0) {
            *reinterpret_cast<__half*>(tile + O4_VS + int4_vmeta_off(s, g)) = sh;
            *reinterpret_cast<__half*>(tile + O4_VM + int4_vmeta_off(s, g)) = mh;
        }
    }
}

// Reads cached tokens back: one CTA per (token, KV head), thread j < 128 key
// channel j, thread 128 + j value channel j; one fp32 fma, one rounding to bf16.
__global__ void __launch_bounds__(256)
dequant_int4_kernel(const uint8_t* __restrict__ cache, int64_t num_pages, int H_kv,
                    const int32_t* __restrict__ slot_mapping, __nv_bfloat16* __restrict__ k_rot,
                    __nv_bfloat16* __restrict__ v_rot) {
    griddep_wait();
    griddep_launch_dependents();
    const int t = blockIdx.x, h = blockIdx.y;
    const int side = threadIdx.x >> 7, j = threadIdx.x & (D - 1);
    __nv_bfloat16* dst = side ? v_rot : k_rot;
    if (!dst) return;
    const int slot = __ldg(slot_mapping + t);
    float val = 0.f;
    if (slot >= 0 && (int64_t)slot < num_pages * PAGE) {
        const int s = slot % PAGE, g = j >> 5;
        const uint8_t* tile = cache + ((size_t)(slot / PAGE) * H_kv + h) * INT4_TILE;
        int code;
        const __half *ps, *pm;
        if (side) {
            const int r = (j >> 2) & 7, i = j & 3;
            code = *reinterpret_cast<const uint16_t*>(tile + O4_VC + 128 * (s >> 1) + 16 * r + 4 * g + 2 * (s & 1)) >> (4 * i);
            ps = reinterpret_cast<const __half*>(tile + O4_VS + int4_vmeta_off(s, g));
            pm = reinterpret_cast<const __half*>(tile + O4_VM + int4_vmeta_off(s, g));
        } else {
            const int tt = (j >> 3) & 3, i = j & 7;
            code = (int)(*reinterpret_cast<const uint32_t*>(tile + O4_KC + 64 * s + 16 * tt + 4 * g) >> (4 * i));
            ps = reinterpret_cast<const __half*>(tile + O4_KM + 16 * s + 2 * g);
            pm = reinterpret_cast<const __half*>(tile + O4_KM + 16 * s + 8 + 2 * g);
        }
        val = __fmaf_rn((float)(code & 15), __half2float(*ps), __half2float(*pm));
    }
    dst[((size_t)t * H_kv + h) * D + j] = __float2bfloat16_rn(val);
}

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_int4_tile_bytes(int d) { return d == D ? (size_t)INT4_TILE : 0; }

extern "C" kvq_status kvq_append_int4(const void* k, const void* v, int n_tok, int H_kv, int d,
                                      const int32_t* slot_mapping, const float* mu_k, const float* R_k,
                                      const float* R_v, float clip, void* cache, int64_t num_pages,
                                      int32_t* err_count, void* stream) {
    if (d != D) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "kvq_append_int4: d=%d (only 128)", d);
    if (n_tok < 0 || H_kv <= 0 || num_pages <= 0)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_append_int4: n_tok=%d H_kv=%d num_pages=%lld", n_tok, H_kv,
                             (long long)num_pages);
    if (H_kv > 65535) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "kvq_append_int4: H_kv=%d too large", H_kv);
    if (!(clip > 0.f && clip <= 1.f))
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_append_int4: clip ratio %g outside (0, 1]", (double)clip);
    if (n_tok == 0) return KVQ_OK;
    if (!k || !v || !slot_mapping || !mu_k || !R_k || !R_v || !cache)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_append_int4: null pointer");
    if (reinterpret_cast<uintptr_t>(cache) % 16)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_append_int4: cache not 16-byte aligned");
    return kvq_check_cuda(launch_pdl(append_int4_kernel, dim3(n_tok, H_kv), dim3(256), 0,
                                     static_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(k),
                                     static_cast<const __nv_bfloat16*>(v), n_tok, H_kv, slot_mapping, mu_k, R_k, R_v,
                                     static_cast<uint8_t*>(cache), num_pages, err_count, clip),
                          "kvq_append_int4 launch");
}

extern "C" kvq_status kvq_dequant_int4(const void* cache, int64_t num_pages, int H_kv, int d,
                                       const int32_t* slot_mapping, int n, void* k_rot, void* v_rot, void* stream) {
    if (d != D) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "kvq_dequant_int4: d=%d (only 128)", d);
    if (n < 0 || H_kv <= 0 || H_kv > 65535 || num_pages <= 0)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_dequant_int4: n=%d H_kv=%d num_pages=%lld", n, H_kv,
                             (long long)num_pages);
    if (n == 0) return KVQ_OK;
    if (!cache || !slot_mapping || (!k_rot && !v_rot))
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_dequant_int4: null pointer");
    if (reinterpret_cast<uintptr_t>(cache) % 16)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_dequant_int4: cache not 16-byte aligned");
    return kvq_check_cuda(launch_pdl(dequant_int4_kernel, dim3(n, H_kv), dim3(256), 0,
                                     static_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(cache), num_pages,
                                     H_kv, slot_mapping, static_cast<__nv_bfloat16*>(k_rot),
                                     static_cast<__nv_bfloat16*>(v_rot)),
                          "kvq_dequant_int4 launch");
}
