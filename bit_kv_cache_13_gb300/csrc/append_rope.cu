// Append to the INT4 cache from a projection's output: the heads' norms of queries and
// keys, the position rotation, and the quantising append of the rotated keys.
//
//   y = x w / sqrt(mean x^2 + eps);  a' = a cos - b sin, b' = b cos + a sin;  bf16(y')
//
// The rotated values are those of the real numbers, rounded once: a cached code depends
// on every bit of the key, so the key must not depend on which kernel formed it.  Fp32
// gives each value to within 2^-19 of its terms; where a rounding to bf16 lies within
// that (one value in a thousand) it is formed again in pairs of fp32 values.
#include <cstddef>

#include "int4_common.cuh"

namespace kvq {

struct RopeArgs {
    const __nv_bfloat16 *q, *k;
    int64_t q_stride, k_stride;
    int n_tok, H_q, H_kv;
    const int32_t* positions;
    const float* table;  // [max_pos][rot]: cos, then sin
    int max_pos, rot;
    const __nv_bfloat16 *q_weight, *k_weight;
    double eps;
    __nv_bfloat16 *q_out, *k_out;
};

constexpr int RP_ROWS = 8;  // heads of a token that a warp takes
constexpr float RP_BOUND = 0x1p-19f;
constexpr float RP_SMALL = 0x1p-80f, RP_LARGE = 0x1p80f;  // fp32 holds products' low parts between these

__device__ __forceinline__ void rope_unpack(uint4 raw, float (&x)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t rope_pack(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// hi + lo, hi the nearest fp32 to it, to the nearest bf16: only where hi is half way between two does lo decide.
__device__ __forceinline__ uint16_t rope_round(float hi, float lo) {
    uint32_t b = __float_as_uint(hi);
    if ((b & 0xffffu) == 0x8000u && lo != 0.f) b += (lo > 0.f) == (hi > 0.f) ? 1u : 0xffffffffu;
    return __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(b)));
}

// The element whose terms are a c - b s (the first of a pair) or a c + b s, times 1 / sqrt(v), in fp64.
__device__ __noinline__ uint16_t rope_wide(double a, double b, float c, float s, double v, bool norm) {
    double y = a * (double)c + b * (double)s;
    if (norm) y *= 1.0 / sqrt(v);
    float f = __double2float_rz(y);
    if (isfinite(f) && (double)f != y) f = __uint_as_float(__float_as_uint(f) | 1u);  // (something is left below it)
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// Row of 16 lanes, eight elements each: those of `open` (one bit an element) are formed again, into out.  a: the
// element, b: its pair's other, negative for the first of a pair (0 beyond the rotated part), without their weights.
__device__ __noinline__ void rope_again(const float (&x)[8], const float (&a)[8], const float (&b)[8], const float (&c)[8],
                                        const float (&s)[8], const float (&wa)[8], const float (&wb)[8], double eps, bool norm,
                                        bool wild, uint32_t open, uint16_t (&out)[8]) {
    Dd r = {1.f, 0.f};
    double v = 1.0;
    if (norm) {
        if (__any_sync(0xffffffffu, wild)) {
            double n2 = 0.0;
            for (int e = 0; e < 8; ++e) n2 = fma((double)x[e], (double)x[e], n2);
            for (int o = 8; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
            v = n2 / D + eps;
        }
        Dd n2 = {0.f, 0.f};
        for (int e = 0; e < 8; ++e) dd_fma(n2, x[e], 0.f, x[e]);
        for (int o = 8; o; o >>= 1) {
            const Dd y = {__shfl_xor_sync(0xffffffffu, n2.hi, o), __shfl_xor_sync(0xffffffffu, n2.lo, o)};
            dd_add(n2, y);
        }
        n2.hi *= 1.f / D;
        n2.lo *= 1.f / D;
        const float eh = (float)eps;
        dd_add(n2, Dd{eh, (float)(eps - (double)eh)});
        n2 = dd_norm(n2);
        if (!wild) v = (double)n2.hi + (double)n2.lo;
        // 1 / sqrt: one step of Newton's method from the fp32 value, its residual exactly
        const float r0 = rsqrtf(n2.hi), p = __fmul_rn(r0, r0), pe = __fmaf_rn(r0, r0, -p);
        const float z = __fmul_rn(n2.hi, p), ze = __fmaf_rn(n2.hi, p, -z);
        const float d = __fsub_rn(1.f, z) - ze - fmaf(n2.hi, pe, n2.lo * p);
        r = {r0, r0 * fmaf(0.375f * d, d, 0.5f * d)};
    }
    for (int e = 0; e < 8; ++e) {
        if (!(open >> e & 1)) continue;
        const float pa = a[e] * wa[e], pb = b[e] * wb[e];  // (exact: two bf16 factors)
        const float m = __fmul_rn(pa, c[e]), n = __fmul_rn(pb, s[e]), top = fabsf(m) + fabsf(n);
        if (wild || !(top > RP_SMALL && top < RP_LARGE && r.hi < RP_LARGE)) {
            out[e] = rope_wide((double)a[e] * wa[e], (double)b[e] * wb[e], c[e], s[e], v, norm);
            continue;
        }
        float hi, lo;
        two_sum(m, n, hi, lo);
        lo += __fmaf_rn(pa, c[e], -m) + __fmaf_rn(pb, s[e], -n);
        const float h = __fmul_rn(hi, r.hi), l = __fmaf_rn(hi, r.hi, -h) + fmaf(hi, r.lo, lo * r.hi);
        float yh, yl;
        two_sum(h, l, yh, yl);
        out[e] = rope_round(yh, yl);
    }
}

// A warp takes RP_ROWS heads of a token, two at a time (16 lanes a head, 16 bytes each).
template <bool INTERLEAVED>
__global__ void __launch_bounds__(128) rope_kernel(const __grid_constant__ RopeArgs a) {
    const int lane = threadIdx.x & 31, l = lane & 15, rows = a.H_q + a.H_kv, groups = (rows + RP_ROWS - 1) / RP_ROWS;
    const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t t = wid / groups;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= a.n_tok) return;
    const int row0 = (int)(wid % groups) * RP_ROWS + (lane >> 4);
    uint4 raw[RP_ROWS / 2];
#pragma unroll
    for (int i = 0; i < RP_ROWS / 2; ++i) {
        const int row = row0 + 2 * i;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows)
            raw[i] = *reinterpret_cast<const uint4*>((row < a.H_q ? a.q + t * a.q_stride + row * D
                                                                  : a.k + t * a.k_stride + (row - a.H_q) * D) + 8 * l);
    }
    const int pos = __ldg(a.positions + t);
    const bool there = (unsigned)pos < (unsigned)a.max_pos;
    const int half = a.rot / 2;
    const bool rotated = 8 * l < a.rot, second = !INTERLEAVED && 8 * l >= half;
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
    }
    if (there && rotated) {
        const float* row = a.table + (size_t)pos * a.rot;
        if constexpr (INTERLEAVED) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(row + 4 * l)), y = __ldg(reinterpret_cast<const float4*>(row + half + 4 * l));
            c[0] = c[1] = x.x, c[2] = c[3] = x.y, c[4] = c[5] = x.z, c[6] = c[7] = x.w;
            s[0] = s[1] = y.x, s[2] = s[3] = y.y, s[4] = s[5] = y.z, s[6] = s[7] = y.w;
        } else {
            row += second ? 8 * l - half : 8 * l;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(row + e)), y = __ldg(reinterpret_cast<const float4*>(row + half + e));
                c[e] = x.x, c[e + 1] = x.y, c[e + 2] = x.z, c[e + 3] = x.w;
                s[e] = y.x, s[e + 1] = y.y, s[e + 2] = y.z, s[e + 3] = y.w;
            }
        }
    }
    // the lane of the pairs' other halves
    const int other = (lane & 16) | (!rotated ? l : second ? l - half / 8 : l + half / 8);
    const float sign = second ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < RP_ROWS / 2; ++i) {
        const int row = row0 + 2 * i;
        const bool is_q = row < a.H_q, live = row < rows;
        const __nv_bfloat16* weight = is_q ? a.q_weight : a.k_weight;
        const bool norm = weight != nullptr;
        float x[8], w[8], p[8];
        rope_unpack(raw[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (norm) rope_unpack(__ldg(reinterpret_cast<const uint4*>(weight + 8 * l)), w);
        float n2 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            n2 = fmaf(x[e], x[e], n2);
            p[e] = x[e] * w[e];
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
        const float v = fmaf(n2, 1.f / D, (float)a.eps);
        const bool wild = norm && !(v > RP_SMALL && v < RP_LARGE);
        const float r = norm ? rsqrtf(v) : 1.f;
        uint32_t open = 0u, lo[4], hi[4];
        float y[8], d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float b;
            if constexpr (INTERLEAVED)
                b = !rotated ? 0.f : e & 1 ? p[e - 1] : -p[e + 1];
            else {
                b = __shfl_sync(0xffffffffu, p[e], other);
                b = rotated ? sign * b : 0.f;
            }
            const float m = p[e] * c[e], n = b * s[e], top = fabsf(m) + fabsf(n);
            y[e] = (m + n) * r;
            d[e] = RP_BOUND * top * r;
            // (0 of factors that are not: what is left below fp32's range)
            if (wild || !((top > RP_SMALL && top < RP_LARGE) || (p[e] == 0.f && b == 0.f))) open |= 1u << e;
            if (p[e] == 0.f && x[e] != 0.f) open |= 0x100u;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo[e] = rope_pack(y[2 * e] - d[2 * e], y[2 * e + 1] - d[2 * e + 1]);
            hi[e] = rope_pack(y[2 * e] + d[2 * e], y[2 * e + 1] + d[2 * e + 1]);
            const uint32_t diff = lo[e] ^ hi[e];
            open |= (diff & 0xffffu ? 1u << (2 * e) : 0u) | (diff >> 16 ? 2u << (2 * e) : 0u);
        }
        // a product that vanished takes its whole head along
        if (__ballot_sync(0xffffffffu, open & 0x100u) >> (lane & 16) & 0xffffu) open = 0xffu;
        if (!live || !there) open = 0u;
        if (__any_sync(0xffffffffu, open)) {
            float b[8], wb[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (INTERLEAVED) {
                    b[e] = e & 1 ? x[e - 1] : -x[e + 1];
                    wb[e] = e & 1 ? w[e - 1] : w[e + 1];
                } else {
                    b[e] = sign * __shfl_sync(0xffffffffu, x[e], other);
                    wb[e] = __shfl_sync(0xffffffffu, w[e], other);
                }
                if (!rotated) b[e] = 0.f, wb[e] = 0.f;
            }
            uint16_t again[8];
            rope_again(x, x, b, c, s, w, wb, a.eps, norm, wild, open, again);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (open >> e & 1) lo[e >> 1] = e & 1 ? (lo[e >> 1] & 0xffffu) | (uint32_t)again[e] << 16 : (lo[e >> 1] & 0xffff0000u) | again[e];
        }
        if (live) {
            __nv_bfloat16* out = is_q ? a.q_out + (t * a.H_q + row) * D : a.k_out + (t * a.H_kv + (row - a.H_q)) * D;
            *reinterpret_cast<uint4*>(out + 8 * l) = there ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

}  // namespace kvq

using namespace kvq;

namespace {

struct Span {
    uintptr_t first, end;
};
Span span(const void* p, int64_t n_tok, int64_t stride, int64_t row) {  // elements of two bytes
    const uintptr_t x = reinterpret_cast<uintptr_t>(p);
    return {x, x + 2 * (uintptr_t)((n_tok - 1) * stride + row)};
}
bool meet(Span a, Span b) { return a.first < b.end && b.first < a.end; }

}  // namespace

extern "C" kvq_status kvq_append_rope_int4(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                           int64_t v_stride, int n_tok, int H_q, int H_kv, int d,
                                           const int32_t* positions, const float* rope, int max_pos, int rot_dim,
                                           int interleaved, const void* q_weight, const void* k_weight, double eps,
                                           const int32_t* slot_mapping, const float* mu_k, const float* R_k,
                                           const float* R_v, float clip, void* cache, int64_t num_pages, void* q_out,
                                           void* k_out, int32_t* err_count, void* stream) {
    const char* fn = "kvq_append_rope_int4";
    if (H_q <= 0 || max_pos <= 0) return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: H_q=%d max_pos=%d", fn, H_q, max_pos);
    if (H_q > 65535) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: H_q=%d too large", fn, H_q);
    if (rot_dim < 16 || rot_dim > D || rot_dim % 16)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: rot_dim=%d is not a multiple of 16 in 16..128", fn, rot_dim);
    if (!(eps >= 0.0 && eps <= 1e30)) return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: eps %g is not within 0 and 1e30", fn, eps);
    AppendInt4 a = {};
    a.k = static_cast<const __nv_bfloat16*>(k_out);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.k_stride = (int64_t)H_kv * D;
    a.v_stride = v_stride;
    a.n_tok = n_tok;
    a.H_kv = H_kv;
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.max_pos = max_pos;
    a.mu_k = mu_k;
    a.R_k = R_k;
    a.R_v = R_v;
    a.clip = clip;
    a.cache = static_cast<uint8_t*>(cache);
    a.num_pages = num_pages;
    a.err_count = err_count;
    kvq_status st = kvq_append_int4_args(fn, a, d);
    if (st != KVQ_OK || n_tok == 0) return st;
    if (!q || !k || !positions || !rope || !q_out) return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void* p : {q, k, (const void*)rope, q_weight, k_weight, (const void*)q_out})
        if (reinterpret_cast<uintptr_t>(p) % 16)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: q, k, rope, the weights and q_out need to be 16-byte aligned", fn);
    const int64_t rows[3] = {(int64_t)H_q * D, (int64_t)H_kv * D, (int64_t)H_kv * D}, strides[3] = {q_stride, k_stride, v_stride};
    for (int i = 0; i < 3; ++i)
        if (strides[i] < rows[i] || strides[i] % 8 || strides[i] > (int64_t(1) << 40) / n_tok)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: a token stride of %lld elements (at least a token's heads, a multiple of 8, "
                                 "2^40 elements in all)", fn, (long long)strides[i]);
    // an output may stand in its input's place, row for row, and nowhere else in what is read
    const Span in[3] = {span(q, n_tok, q_stride, rows[0]), span(k, n_tok, k_stride, rows[1]), span(v, n_tok, v_stride, rows[2])};
    const Span out[2] = {span(q_out, n_tok, rows[0], rows[0]), span(k_out, n_tok, rows[1], rows[1])};
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 3; ++i)
            if (meet(out[o], in[i]) && !(o == i && out[o].first == in[i].first && out[o].end == in[i].end))
                return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: q_out or k_out overlaps q, k or v other than in place", fn);
    if (meet(out[0], out[1])) return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: q_out overlaps k_out", fn);
    RopeArgs r;
    r.q = static_cast<const __nv_bfloat16*>(q);
    r.k = static_cast<const __nv_bfloat16*>(k);
    r.q_stride = q_stride;
    r.k_stride = k_stride;
    r.n_tok = n_tok;
    r.H_q = H_q;
    r.H_kv = H_kv;
    r.positions = positions;
    r.table = rope;
    r.max_pos = max_pos;
    r.rot = rot_dim;
    r.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
    r.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
    r.eps = eps;
    r.q_out = static_cast<__nv_bfloat16*>(q_out);
    r.k_out = static_cast<__nv_bfloat16*>(k_out);
    const int64_t warps = (int64_t)n_tok * ((H_q + H_kv + RP_ROWS - 1) / RP_ROWS), blocks = (warps + 3) / 4;
    if (blocks > 0x7fffffff) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: n_tok * (H_q + H_kv) too large", fn);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    st = kvq_check_cuda(launch_pdl(interleaved ? rope_kernel<true> : rope_kernel<false>, dim3((unsigned)blocks), dim3(128), 0, cs, r),
                        "kvq_append_rope_int4 rotate launch");
    if (st != KVQ_OK) return st;
    return kvq_append_int4_launch("kvq_append_rope_int4 launch", a, cs);
}
