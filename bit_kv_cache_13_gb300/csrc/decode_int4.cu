// Fused packed-cache decode attention over the rotated INT4 cache, and the
// form that accumulates the attention weight each token drew.
//
//   q' = q R_k;  a_s = <q', K^_s> scale;  p = softmax(a);  o = (sum_s p_s V^_s) R_v^T
//
// The context of a (sequence, KV head) is cut into splits of whole pages, one
// CTA each; a split publishes its running maximum, sum and unnormalised
// output, and the last to finish merges them by the log-sum-exp rule, rotates
// the merged output once and writes it.
#include "int4_common.cuh"

namespace kvq {

constexpr int D4_NW = 4;           // warps of a split's CTA
constexpr int D4_MAX_SPLITS = 254;

__device__ __forceinline__ float d4_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct D4Args {
    const __nv_bfloat16* q;
    int B, H_q, H_kv, G;
    const uint8_t* cache;
    int64_t num_pages;
    const int32_t* block_table;
    int max_pages;
    const int32_t* context_lens;
    const float *Rk, *Rv;
    float scale_log2;
    __nv_bfloat16* out;
    uint8_t* ws;
    float* partials;   // [unit][split][G][PART_STRIDE]
    float* logits;     // [unit][16 max_pages][G], base 2 (weights form), else null
    float2* stats;     // [unit][G] (maximum, 1 / sum)
    int S;
};

// Lane l of a warp holds channels 4 l .. 4 l + 3.  Each warp takes every
// fourth page of its split, token by token.
template <int MAXG>
__global__ void __launch_bounds__(D4_NW * 32) decode_int4_kernel(const D4Args a) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float qin[MAXG][D], qr[MAXG][D], op[D4_NW][MAXG][D], mp[D4_NW][MAXG], lp[D4_NW][MAXG];
    __shared__ int last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z, G = a.G;
    const int64_t unit = (int64_t)b * a.H_kv + h;
    const int ctx = max(0, min(__ldg(a.context_lens + b), a.max_pages * PAGE));
    const int pages = (ctx + PAGE - 1) / PAGE, per = (pages + a.S - 1) / a.S;
    const int p0 = min(pages, split * per), p1 = min(pages, p0 + per);
    const __nv_bfloat16* qb = a.q + ((size_t)b * a.H_q + (size_t)h * G) * D;
    for (int i = tid; i < MAXG * D; i += D4_NW * 32) qin[i / D][i % D] = i < G * D ? __bfloat162float(qb[i]) : 0.f;
    __syncthreads();
    {
        const float* R = a.Rk + (size_t)h * D * D + tid;  // thread = channel
        float acc[MAXG];
#pragma unroll
        for (int j = 0; j < MAXG; ++j) acc[j] = 0.f;
        for (int i = 0; i < D; ++i) {
            const float r = __ldg(R + (size_t)i * D);
#pragma unroll
            for (int j = 0; j < MAXG; ++j) acc[j] = fmaf(qin[j][i], r, acc[j]);
        }
#pragma unroll
        for (int j = 0; j < MAXG; ++j) qr[j][tid] = acc[j] * a.scale_log2;
    }
    __syncthreads();
    float m[MAXG], l[MAXG], o[MAXG][4];
#pragma unroll
    for (int j = 0; j < MAXG; ++j) {
        m[j] = -CUDART_INF_F;
        l[j] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    }
    const int g = lane >> 3;
    for (int p = p0 + warp; p < p1; p += D4_NW) {
        const int pid = __ldg(a.block_table + (size_t)b * a.max_pages + p);
        const bool bad = pid < 0 || (int64_t)pid >= a.num_pages;
        if (bad && lane == 0) atomicOr(reinterpret_cast<uint32_t*>(a.ws), ERR_BAD_PAGE);
        const uint8_t* tile = a.cache + ((size_t)(bad ? 0 : pid) * a.H_kv + h) * INT4_TILE;
        const int n = min(PAGE, ctx - p * PAGE);
        for (int s = 0; s < n; ++s) {
            float lg[MAXG];
            if (bad) {
#pragma unroll
                for (int j = 0; j < MAXG; ++j) lg[j] = -CUDART_INF_F;
            } else {
                const int t = (lane >> 1) & 3;
                const uint32_t kc = *reinterpret_cast<const uint16_t*>(tile + O4_KC + 64 * s + 16 * t + 4 * g + 2 * (lane & 1));
                const float ks = __half2float(*reinterpret_cast<const __half*>(tile + O4_KM + 16 * s + 2 * g));
                const float km = __half2float(*reinterpret_cast<const __half*>(tile + O4_KM + 16 * s + 8 + 2 * g));
                const uint32_t vc = *reinterpret_cast<const uint16_t*>(tile + O4_VC + 128 * (s >> 1) + 16 * (lane & 7) + 4 * g + 2 * (s & 1));
                const float vs = __half2float(*reinterpret_cast<const __half*>(tile + O4_VS + int4_vmeta_off(s, g)));
                const float vm = __half2float(*reinterpret_cast<const __half*>(tile + O4_VM + int4_vmeta_off(s, g)));
                float kv[4], vv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    kv[e] = fmaf((float)((kc >> (4 * e)) & 15), ks, km);
                    vv[e] = fmaf((float)((vc >> (4 * e)) & 15), vs, vm);
                }
#pragma unroll
                for (int j = 0; j < MAXG; ++j) {
                    const float* qq = &qr[j][4 * lane];
                    float d = fmaf(qq[0], kv[0], fmaf(qq[1], kv[1], fmaf(qq[2], kv[2], qq[3] * kv[3])));
#pragma unroll
                    for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
                    lg[j] = d;
                    const float mn = fmaxf(m[j], d), c = d4_ex2(m[j] - mn), pw = d4_ex2(d - mn);
                    l[j] = fmaf(l[j], c, pw);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][e] = fmaf(o[j][e], c, pw * vv[e]);
                    m[j] = mn;
                }
            }
            if (a.logits && lane == 0)
                for (int j = 0; j < G; ++j)
                    a.logits[((size_t)unit * a.max_pages * PAGE + (size_t)p * PAGE + s) * G + j] = lg[j];
        }
    }
#pragma unroll
    for (int j = 0; j < MAXG; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) op[warp][j][4 * lane + e] = o[j][e];
        if (lane == 0) {
            mp[warp][j] = m[j];
            lp[warp][j] = l[j];
        }
    }
    __syncthreads();
    float* part = a.partials + ((size_t)unit * a.S + split) * G * PART_STRIDE;
    for (int j = 0; j < G; ++j) {
        float M = -CUDART_INF_F, L = 0.f, O = 0.f;
        for (int w = 0; w < D4_NW; ++w) M = fmaxf(M, mp[w][j]);
        for (int w = 0; w < D4_NW; ++w) {
            const float f = M == -CUDART_INF_F ? 0.f : d4_ex2(mp[w][j] - M);
            L = fmaf(lp[w][j], f, L);
            O = fmaf(op[w][j][tid], f, O);
        }
        part[(size_t)j * PART_STRIDE + 4 + tid] = O;
        if (tid == 0) {
            part[(size_t)j * PART_STRIDE] = M;
            part[(size_t)j * PART_STRIDE + 1] = L;
        }
    }
    __syncthreads();
    int32_t* ticket = reinterpret_cast<int32_t*>(a.ws + WS_HEADER) + unit;
    if (tid == 0) last = atomic_add_acq_rel_gpu(ticket, 1) == a.S - 1;
    __syncthreads();
    if (!last) return;
    // merge, normalise, rotate by R_v^T
    const float* pu = a.partials + (size_t)unit * a.S * G * PART_STRIDE;
    for (int j = 0; j < G; ++j) {
        float M = -CUDART_INF_F, L = 0.f, O = 0.f;
        for (int s = 0; s < a.S; ++s) M = fmaxf(M, __ldcg(pu + ((size_t)s * G + j) * PART_STRIDE));
        for (int s = 0; s < a.S; ++s) {
            const float* ps = pu + ((size_t)s * G + j) * PART_STRIDE;
            const float f = M == -CUDART_INF_F ? 0.f : d4_ex2(__ldcg(ps) - M);
            L = fmaf(__ldcg(ps + 1), f, L);
            O = fmaf(__ldcg(ps + 4 + tid), f, O);
        }
        qin[j][tid] = L > 0.f ? O / L : (L == L ? 0.f : L);
        if (a.stats && tid == 0) a.stats[unit * G + j] = make_float2(M, L > 0.f ? 1.f / L : (L == L ? 0.f : L));
    }
    __syncthreads();
    for (int j = 0; j < G; ++j) {
        const float* R = a.Rv + ((size_t)h * D + tid) * D;
        float acc = 0.f;
        for (int c = 0; c < D; ++c) acc = fmaf(qin[j][c], __ldg(R + c), acc);
        a.out[((size_t)b * a.H_q + (size_t)h * G + j) * D + tid] = __float2bfloat16_rn(acc);
    }
    if (tid == 0) *ticket = 0;
}

// weights[s] = decay weights[s] + sum_j 2^(a_{j,s} - M_j) / L_j: reads the
// logits that the attention kernel stored.
__global__ void __launch_bounds__(256)
weights_int4_kernel(const float* __restrict__ logits, const float2* __restrict__ stats, int H_kv, int G, int max_pages,
                    const int32_t* __restrict__ context_lens, float* __restrict__ weights, int64_t stride, float decay) {
    griddep_wait();
    griddep_launch_dependents();
    const int h = blockIdx.y, b = blockIdx.z;
    const int64_t unit = (int64_t)b * H_kv + h;
    const int ctx = max(0, min(__ldg(context_lens + b), max_pages * PAGE));
    const float2* st = stats + unit * G;
    for (int64_t s = (int64_t)blockIdx.x * 256 + threadIdx.x; s < ctx; s += (int64_t)gridDim.x * 256) {
        const float* lg = logits + ((size_t)unit * max_pages * PAGE + s) * G;
        float p = 0.f;
        for (int j = 0; j < G; ++j) {
            const float2 ml = __ldcg(st + j);
            const float x = __ldcg(lg + j);
            // (a dropped token's logit is -inf: no weight, whatever the maximum)
            p += x == -CUDART_INF_F ? 0.f : d4_ex2(x - ml.x) * ml.y;
        }
        float* w = weights + unit * stride + s;
        *w = fmaf(decay, *w, p);
    }
}

}  // namespace kvq

using namespace kvq;

// Splits per unit: about four CTAs per SM in all, at least four pages each.
static int d4_splits(int B, int H_kv, int max_pages, int num_splits) {
    int64_t s = num_splits > 0 ? num_splits : (int64_t)kvq_device_sm_count() * 4 / ((int64_t)B * H_kv);
    const int64_t cap = (max_pages + 3) / 4;
    if (num_splits <= 0 && s > cap) s = cap;
    if (s > D4_MAX_SPLITS) s = D4_MAX_SPLITS;
    return s < 1 ? 1 : (int)s;
}

struct D4Layout {
    size_t partials, stats, logits, total;
};
static D4Layout d4_layout(int B, int H_q, int H_kv, int max_pages, int S, bool weights) {
    const size_t units = (size_t)B * H_kv, G = (size_t)(H_q / H_kv);
    D4Layout l;
    l.partials = WS_HEADER + tickets_bytes(B, H_kv);
    l.stats = align_up(l.partials + units * S * G * PART_STRIDE * 4, 256);
    l.logits = align_up(l.stats + (weights ? units * G * 8 : 0), 256);
    l.total = l.logits + (weights ? units * (size_t)max_pages * PAGE * G * 4 : 0);
    return l;
}

extern "C" size_t kvq_int4_workspace_bytes(int B, int H_q, int H_kv, int max_pages_per_seq, int num_splits,
                                           int weights) {
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || max_pages_per_seq <= 0 || max_pages_per_seq >= (1 << 27) ||
        num_splits < 0 || num_splits > D4_MAX_SPLITS || B > 65535 || H_kv > 65535)
        return 0;
    return d4_layout(B, H_q, H_kv, max_pages_per_seq, d4_splits(B, H_kv, max_pages_per_seq, num_splits), weights != 0).total;
}

static kvq_status decode_int4(const char* fn, const void* q, int B, int H_q, int H_kv, int d, const void* cache,
                              int64_t num_pages, const int32_t* block_table, int max_pages,
                              const int32_t* context_lens, const float* R_k, const float* R_v, float scale, void* out,
                              bool with_weights, float* weights, int64_t weights_stride, float decay, void* workspace,
                              size_t workspace_bytes, int num_splits, void* stream) {
    if (d != D) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: d=%d (only 128)", fn, d);
    if (B <= 0 || H_kv <= 0 || H_q <= 0 || H_q % H_kv || max_pages <= 0 || num_pages <= 0 || num_splits < 0)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: B=%d H_q=%d H_kv=%d max_pages=%d num_pages=%lld splits=%d", fn,
                             B, H_q, H_kv, max_pages, (long long)num_pages, num_splits);
    const int G = H_q / H_kv;
    if (G > 8) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: GQA group %d > 8", fn, G);
    if (B > 65535 || H_kv > 65535) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: B or H_kv above 65535", fn);
    if (max_pages >= (1 << 27))
        return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: max_pages_per_seq %d not below 2^27", fn, max_pages);
    if (num_splits > D4_MAX_SPLITS)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: %d splits above %d", fn, num_splits, D4_MAX_SPLITS);
    if (!q || !cache || !block_table || !context_lens || !R_k || !R_v || !out || !workspace || (with_weights && !weights))
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void* p : {q, cache, (const void*)R_k, (const void*)R_v, (const void*)out, (const void*)workspace})
        if (reinterpret_cast<uintptr_t>(p) % 16)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: q, cache, R_k, R_v, out and workspace need 16-byte alignment", fn);
    if (with_weights) {
        if (weights_stride < (int64_t)max_pages * PAGE)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: weights_stride %lld below 16 * max_pages_per_seq", fn,
                                 (long long)weights_stride);
        if (!(decay >= 0.f && decay <= 3.402823466e38f))
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: decay %g is not finite and >= 0", fn, (double)decay);
    }
    const int S = d4_splits(B, H_kv, max_pages, num_splits);
    const D4Layout lay = d4_layout(B, H_q, H_kv, max_pages, S, with_weights);
    if (workspace_bytes < lay.total)
        return kvq_set_error(KVQ_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, workspace_bytes, lay.total);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    D4Args a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.B = B;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.G = G;
    a.cache = static_cast<const uint8_t*>(cache);
    a.num_pages = num_pages;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.context_lens = context_lens;
    a.Rk = R_k;
    a.Rv = R_v;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.ws = ws;
    a.partials = reinterpret_cast<float*>(ws + lay.partials);
    a.stats = with_weights ? reinterpret_cast<float2*>(ws + lay.stats) : nullptr;
    a.logits = with_weights ? reinterpret_cast<float*>(ws + lay.logits) : nullptr;
    a.S = S;
    const kvq_status st = kvq_check_cuda(launch_pdl(G <= 4 ? decode_int4_kernel<4> : decode_int4_kernel<8>, dim3(S, H_kv, B),
                                                    dim3(D4_NW * 32), 0, static_cast<cudaStream_t>(stream), a),
                                         "kvq_decode_attn_int4 launch");
    if (st != KVQ_OK || !with_weights) return st;
    const int gx = (max_pages * PAGE + 255) / 256;
    return kvq_check_cuda(launch_pdl(weights_int4_kernel, dim3(gx < 64 ? gx : 64, H_kv, B), dim3(256), 0,
                                     static_cast<cudaStream_t>(stream), (const float*)a.logits, (const float2*)a.stats,
                                     H_kv, G, max_pages, context_lens, weights, weights_stride, decay),
                          "kvq_decode_attn_int4_weights launch");
}

extern "C" kvq_status kvq_decode_attn_int4(const void* q, int B, int H_q, int H_kv, int d, const void* cache,
                                           int64_t num_pages, const int32_t* block_table, int max_pages_per_seq,
                                           const int32_t* context_lens, const float* R_k, const float* R_v,
                                           float scale, void* out, void* workspace, size_t workspace_bytes,
                                           int num_splits, void* stream) {
    return decode_int4("kvq_decode_attn_int4", q, B, H_q, H_kv, d, cache, num_pages, block_table, max_pages_per_seq,
                       context_lens, R_k, R_v, scale, out, false, nullptr, 0, 0.f, workspace, workspace_bytes,
                       num_splits, stream);
}

extern "C" kvq_status kvq_decode_attn_int4_weights(const void* q, int B, int H_q, int H_kv, int d, const void* cache,
                                                   int64_t num_pages, const int32_t* block_table,
                                                   int max_pages_per_seq, const int32_t* context_lens,
                                                   const float* R_k, const float* R_v, float scale, void* out,
                                                   float* weights, int64_t weights_stride, float decay,
                                                   void* workspace, size_t workspace_bytes, int num_splits,
                                                   void* stream) {
    return decode_int4("kvq_decode_attn_int4_weights", q, B, H_q, H_kv, d, cache, num_pages, block_table,
                       max_pages_per_seq, context_lens, R_k, R_v, scale, out, true, weights, weights_stride, decay,
                       workspace, workspace_bytes, num_splits, stream);
}
