// Append to the INT4 cache from a projection's output: the heads' norms of queries and
// keys, the position rotation, and the quantising append of the rotated keys.
//
//   y = x w / sqrt(mean x^2 + eps);  a' = a cos - b sin, b' = b cos + a sin;  bf16(y')
//
// The rotated values are those of the real numbers, rounded once: a cached code depends
// on every bit of the key, so the key must not depend on which kernel formed it.  Fp32
// gives each value to within 2^-20 of its terms; where a rounding to bf16 lies within
// that (one value in a thousand or two) it is formed again in pairs of fp32 values, which
// leave less than 2^-42 of the terms: the mean of squares 2^-43.5 (seven additions of low
// parts, four across lanes), halved by the root, and 2^-46 each for Newton's step, the
// root's low part and the product's.
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
    int per;  // heads of a token that a warp takes
};

// Of a value's terms |a cos| + |b sin|, in units of 2^-24: the sum of squares 9 (4 and 1 additions, 4 across lanes) and the
// mean's 1, halved by the root; the root 1.5 after its step of Newton's method; each term, their sum, the product with the
// root and the bound's own sum 1 each: 10.5.
constexpr float RP_BOUND = 10.5f * 0x1p-24f;
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

// (a c + b s) / sqrt(v) in fp64.
__device__ __noinline__ uint16_t rope_wide(double a, double b, float c, float s, double v, bool norm) {
    double y = a * (double)c + b * (double)s;
    if (norm) y *= 1.0 / sqrt(v);
    float f = __double2float_rz(y);
    if (isfinite(f) && (double)f != y) f = __uint_as_float(__float_as_uint(f) | 1u);  // (something is left below it)
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// 1 / sqrt(mean x^2 + eps) of a row of 16 lanes, in a pair (every lane of the warp takes part).
__device__ __forceinline__ Dd rope_root(const float (&x)[8], double eps) {
    Dd n2 = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // (squares of bf16 numbers are exact)
        float t;
        two_sum(n2.hi, __fmul_rn(x[e], x[e]), n2.hi, t);
        n2.lo += t;
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) {
        const Dd y = {__shfl_xor_sync(0xffffffffu, n2.hi, o), __shfl_xor_sync(0xffffffffu, n2.lo, o)};
        dd_add(n2, y);
    }
    n2.hi *= 1.f / D;
    n2.lo *= 1.f / D;
    const float eh = (float)eps;
    dd_add(n2, Dd{eh, (float)(eps - (double)eh)});
    n2 = dd_norm(n2);
    // one step of Newton's method from the fp32 value, its residual exactly
    const float r0 = rsqrtf(n2.hi), p = __fmul_rn(r0, r0), pe = __fmaf_rn(r0, r0, -p);
    const float z = __fmul_rn(n2.hi, p), ze = __fmaf_rn(n2.hi, p, -z);
    const float d = __fsub_rn(1.f, z) - ze - fmaf(n2.hi, pe, n2.lo * p);
    return {r0, r0 * fmaf(0.375f * d, d, 0.5f * d)};
}

// (pa c + pb s) times the root, rounded once.
__device__ __forceinline__ uint16_t rope_value(float pa, float pb, float c, float s, Dd r) {
    const float m = __fmul_rn(pa, c), n = __fmul_rn(pb, s);
    float hi, lo;
    two_sum(m, n, hi, lo);
    lo += __fmaf_rn(pa, c, -m) + __fmaf_rn(pb, s, -n);
    const float h = __fmul_rn(hi, r.hi), l = __fmaf_rn(hi, r.hi, -h) + fmaf(hi, r.lo, lo * r.hi);
    float yh, yl;
    two_sum(h, l, yh, yl);
    return rope_round(yh, yl);
}

// Row of 16 lanes, eight elements each: those of `open` (one bit an element) are formed again, into out.  a: the
// element, b: its pair's other (0 beyond the rotated part), without their weights.
__device__ __noinline__ void rope_again(const float (&x)[8], const float (&a)[8], const float (&b)[8], const float (&c)[8],
                                        const float (&s)[8], const float (&wa)[8], const float (&wb)[8], double eps, bool norm,
                                        bool wild, uint32_t open, uint16_t (&out)[8]) {
    Dd r = {1.f, 0.f};
    double v = 1.0;
    if (__any_sync(0xffffffffu, norm)) {  // (the other half of the warp may hold a head without one)
        double n2 = 0.0;
        for (int e = 0; e < 8; ++e) n2 = fma((double)x[e], (double)x[e], n2);
        for (int o = 8; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
        const Dd root = rope_root(x, eps);
        if (norm) {
            v = n2 / D + eps;
            r = root;
        }
    }
    for (int e = 0; e < 8; ++e) {
        if (!(open >> e & 1)) continue;
        const float pa = a[e] * wa[e], pb = b[e] * wb[e], top = fabsf(pa * c[e]) + fabsf(pb * s[e]);
        if (wild || !(top > RP_SMALL && top < RP_LARGE && r.hi < RP_LARGE))
            out[e] = rope_wide((double)a[e] * wa[e], (double)b[e] * wb[e], c[e], s[e], v, norm);
        else
            out[e] = rope_value(pa, pb, c[e], s[e], r);
    }
}

// Two fp32 operations in one instruction.
#define ROPE_OP2(name, op)                                                                                              \
    __device__ __forceinline__ float2 name(float2 a, float2 b) {                                                        \
        float2 d;                                                                                                       \
        asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n " op ".rn.f32x2 x, x, y;\n"           \
            " mov.b64 {%0, %1}, x;\n}\n"                                                                                \
            : "=f"(d.x), "=f"(d.y)                                                                                      \
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                                                                  \
        return d;                                                                                                       \
    }
ROPE_OP2(rope_mul2, "mul")
ROPE_OP2(rope_add2, "add")
__device__ __forceinline__ float2 rope_fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n fma.rn.f32x2 x, x, y, z;\n"
        " mov.b64 {%0, %1}, x;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// A warp takes `per` heads of a token, two at a time (16 lanes a head, 16 bytes each).  8192 tokens of
// 32 + 8 heads: 77 us, 168 MB (25 us at the copy rate).  Bound by 358 instructions a head pair, most of them for the bound on
// the rounding, and by waits for loads between them: 62 % of the issue slots are taken, long scoreboard is the largest stall.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(128, 6) rope_kernel(const __grid_constant__ RopeArgs a) {
    const int lane = threadIdx.x & 31, l = lane & 15, rows = a.H_q + a.H_kv, groups = (rows + a.per - 1) / a.per;
    const int64_t wid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t t = wid / groups;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= a.n_tok) return;
    const int row0 = (int)(wid % groups) * a.per + (lane >> 4), pairs = a.per / 2;
    // (a token's heads, the keys' behind the queries')
    const __nv_bfloat16 *q_in = a.q + t * a.q_stride + 8 * l, *k_in = a.k + t * a.k_stride - a.H_q * D + 8 * l;
    __nv_bfloat16 *q_to = a.q_out + t * a.H_q * D + 8 * l, *k_to = a.k_out + (t * a.H_kv - a.H_q) * D + 8 * l;
    auto fetch = [&](int row) {
        return row < rows ? *reinterpret_cast<const uint4*>((row < a.H_q ? q_in : k_in) + row * D) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 raw = fetch(row0), raw1 = pairs > 1 ? fetch(row0 + 2) : make_uint4(0u, 0u, 0u, 0u);
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
    // the sines with the signs of the pairs' halves: a cos - b sin, b cos + a sin
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (INTERLEAVED ? !(e & 1) : !second) s[e] = -s[e];
    // (one loop body: the code of four heads side by side does not stay in the instruction cache, 8192 tokens 183 us)
#pragma unroll 1
    for (int i = 0; i < pairs; ++i) {
        const int row = row0 + 2 * i;
        const uint4 raw2 = i + 2 < pairs ? fetch(row + 4) : make_uint4(0u, 0u, 0u, 0u);
        const bool is_q = row < a.H_q, live = row < rows;
        const __nv_bfloat16* weight = is_q ? a.q_weight : a.k_weight;
        const bool norm = weight != nullptr;
        float x[8], w[8], p[8];
        rope_unpack(raw, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (norm) rope_unpack(__ldg(reinterpret_cast<const uint4*>(weight + 8 * l)), w);
        float2 sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            sq = rope_fma2(make_float2(x[e], x[e + 1]), make_float2(x[e], x[e + 1]), sq);
            const float2 y = rope_mul2(make_float2(x[e], x[e + 1]), make_float2(w[e], w[e + 1]));
            p[e] = y.x;
            p[e + 1] = y.y;
        }
        float n2 = sq.x + sq.y;
#pragma unroll
        for (int o = 8; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
        const float v = fmaf(n2, 1.f / D, (float)a.eps);
        const bool wild = norm && !(v > RP_SMALL && v < RP_LARGE);
        float r = 1.f;
        if (norm) {
            r = rsqrtf(v);
            r = fmaf(0.5f * r, fmaf(-v * r, r, 1.f), r);
        }
        uint32_t lo[4], hi[4], differ = 0u, least = 0xffffffffu, most = 0u;
        float pb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            pb[e] = INTERLEAVED ? p[e ^ 1] : __shfl_sync(0xffffffffu, p[e], other);
            if (!rotated) pb[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 m = rope_mul2(make_float2(p[e], p[e + 1]), make_float2(c[e], c[e + 1]));
            const float2 n = rope_mul2(make_float2(pb[e], pb[e + 1]), make_float2(s[e], s[e + 1]));
            const float2 z = rope_add2(m, n), y = rope_mul2(z, make_float2(r, r));
            const float2 d = rope_mul2(make_float2(fabsf(m.x) + fabsf(n.x), fabsf(m.y) + fabsf(n.y)), make_float2(RP_BOUND * r, RP_BOUND * r));
            const float2 up = rope_add2(y, d), down = rope_add2(y, make_float2(-d.x, -d.y));
            lo[e >> 1] = rope_pack(down.x, down.y);
            hi[e >> 1] = rope_pack(up.x, up.y);
            differ |= lo[e >> 1] ^ hi[e >> 1];
            const uint32_t zx = __float_as_uint(z.x) & 0x7fffffffu, zy = __float_as_uint(z.y) & 0x7fffffffu;
            least = min(least, min(zx, zy));
            most = max(most, max(zx, zy));
        }
        const bool edge = wild || least < __float_as_uint(RP_SMALL) || most > __float_as_uint(RP_LARGE);
        if (__any_sync(0xffffffffu, (edge || differ) && live && there)) {
            uint32_t open = 0u, wide = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t diff = lo[e] ^ hi[e];
                open |= (diff & 0xffffu ? 1u << (2 * e) : 0u) | (diff >> 16 ? 2u << (2 * e) : 0u);
            }
            if (__any_sync(0xffffffffu, edge)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {  // (0 of factors that are not: what is left below fp32's range)
                    const float top = fabsf(p[e] * c[e]) + fabsf(pb[e] * s[e]);
                    if (wild || !((top > RP_SMALL && top < RP_LARGE) || (p[e] == 0.f && pb[e] == 0.f)) || (p[e] == 0.f && x[e] != 0.f)) wide = 1u;
                }
            }
            if (!live || !there) open = wide = 0u;
            if (__any_sync(0xffffffffu, wide)) {  // numbers next to fp32's ends: the whole head the long way
                open = __ballot_sync(0xffffffffu, wide) >> (lane & 16) & 0xffffu ? 0xffu : open;
                float xa[8], wa[8], xb[8], wb[8], ca[8], sa[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xa[e] = x[e];
                    wa[e] = w[e];
                    ca[e] = c[e];
                    sa[e] = s[e];
                    xb[e] = INTERLEAVED ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], other);
                    wb[e] = INTERLEAVED ? w[e ^ 1] : __shfl_sync(0xffffffffu, w[e], other);
                    if (!rotated) xb[e] = 0.f, wb[e] = 0.f;
                }
                uint16_t again[8];
                rope_again(xa, xa, xb, ca, sa, wa, wb, a.eps, norm, wild, open, again);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (open >> e & 1) lo[e >> 1] = e & 1 ? (lo[e >> 1] & 0xffffu) | (uint32_t)again[e] << 16 : (lo[e >> 1] & 0xffff0000u) | again[e];
            } else {  // of the products, which are exact, in pairs
                Dd root = {1.f, 0.f};
                if (__any_sync(0xffffffffu, norm)) {  // (of two heads one may have none, a query's last beside a key's first)
                    const Dd y = rope_root(x, a.eps);
                    if (norm) root = y;
                }
                while (open) {
                    const int e = __ffs(open) - 1;
                    open &= open - 1u;
                    float ya = p[0], yb = pb[0], yc = c[0], ys = s[0];
#pragma unroll
                    for (int i = 1; i < 8; ++i)
                        if (e == i) ya = p[i], yb = pb[i], yc = c[i], ys = s[i];
                    const uint32_t v = rope_value(ya, yb, yc, ys, root);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (e == i) lo[i >> 1] = i & 1 ? (lo[i >> 1] & 0xffffu) | v << 16 : (lo[i >> 1] & 0xffff0000u) | v;
                }
                __syncwarp();
            }
        }
        if (live) {
            *reinterpret_cast<uint4*>((is_q ? q_to : k_to) + row * D) = there ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(0u, 0u, 0u, 0u);
        }
        raw = raw1;
        raw1 = raw2;
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
    // Eight heads a warp read their token's row of the table once, but a few tokens are quicker with two (one token of
    // 32 + 8 heads, with the append and the read-back, 15.5 against 17.5 us; 8192 tokens 220 against 168).
    r.per = (int64_t)n_tok * (H_q + H_kv) <= 32 * (int64_t)kvq_device_sm_count() ? 2 : 8;
    const int64_t warps = (int64_t)n_tok * ((H_q + H_kv + r.per - 1) / r.per), blocks = (warps + 3) / 4;
    if (blocks > 0x7fffffff) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: n_tok * (H_q + H_kv) too large", fn);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    st = kvq_check_cuda(launch_pdl(interleaved ? rope_kernel<true> : rope_kernel<false>, dim3((unsigned)blocks), dim3(128), 0, cs, r),
                        "kvq_append_rope_int4 rotate launch");
    if (st != KVQ_OK) return st;
    return kvq_append_int4_launch("kvq_append_rope_int4 launch", a, cs);
}
