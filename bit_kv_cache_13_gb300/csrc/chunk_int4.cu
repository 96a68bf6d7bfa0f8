// Attention of each sequence's last tokens over the rotated INT4 cache: a piece of a
// prompt, drafted tokens, or a whole prompt, causal among themselves, with an optional
// sliding window and sinks.
//
//   q' = q R_k;  a_t = <q', K^_t> scale over the tokens that the query's position sees;
//   o = (sum_t softmax(a)_t V^_t) R_v^T
//
// Rows of 32 (token, head) pairs of one KV head per CTA, a page of 16 tokens at a time,
// all in fp32: four threads a row, four tokens' logits and 32 channels of the output each.
#include <cstddef>

#include "int4_common.cuh"

namespace kvq {

struct ChunkArgs {
    const __nv_bfloat16* q;
    int n_tok;
    const int32_t* q_start;
    int B, H_q, H_kv, G;
    const uint8_t* cache;
    int64_t num_pages;
    const int32_t* block_table;
    int max_pages;
    const int32_t* context_lens;
    const float *Rk, *Rv;
    float scale_log2;
    int window, sinks;
    __nv_bfloat16* out;
    uint32_t* error;
};

constexpr int CH_ROWS = 32;

// New tokens of sequence b: first row and count (0 where q_start is not what it should be).
__device__ __forceinline__ int2 chunk_rows(const ChunkArgs& a, int b) {
    const int s = __ldg(a.q_start + b), e = __ldg(a.q_start + b + 1);
    if (s < 0 || e < s || e > a.n_tok) {
        atomicOr(a.error, ERR_BAD_ROWS);
        return make_int2(0, 0);
    }
    return make_int2(s, e - s);
}

__global__ void __launch_bounds__(128) chunk_int4_kernel(const __grid_constant__ ChunkArgs a) {
    __shared__ __align__(16) float qs[CH_ROWS][D + 4], K[PAGE][D + 4], V[PAGE][D + 4];
    const int tid = threadIdx.x, row = tid >> 2, part = tid & 3, h = blockIdx.y, G = a.G;
    griddep_wait();
    griddep_launch_dependents();
    int b = 0, first = 0;
    int2 rows;
    int64_t block = blockIdx.x;
    for (; b < a.B; ++b) {
        rows = chunk_rows(a, b);
        const int64_t blocks = ((int64_t)rows.y * G + CH_ROWS - 1) / CH_ROWS;
        if (block < blocks) break;
        block -= blocks;
    }
    if (b == a.B) return;
    first = (int)(block * CH_ROWS);
    const int n_rows = (int)min((int64_t)CH_ROWS, (int64_t)rows.y * G - first);
    const int ctx = (int)min((int64_t)max(0, __ldg(a.context_lens + b)), (int64_t)a.max_pages * PAGE);
    const bool live = row < n_rows;
    const int tok = (first + (live ? row : 0)) / G, head = h * G + (first + (live ? row : 0)) % G;
    const int pos = ctx - rows.y + tok;
    // q' into qs
    const __nv_bfloat16* q = a.q + ((size_t)(rows.x + tok) * a.H_q + head) * D;
    float acc[32];
    for (int c = 0; c < 32; ++c) acc[c] = 0.f;
    for (int i = 0; i < D; ++i) {
        const float x = __bfloat162float(q[i]) * a.scale_log2;
        for (int c = 0; c < 32; ++c) acc[c] = fmaf(x, __ldg(a.Rk + ((size_t)h * D + i) * D + 32 * part + c), acc[c]);
    }
    for (int c = 0; c < 32; ++c) qs[row][32 * part + c] = live ? acc[c] : 0.f;
    float m = -CUDART_INF_F, l = 0.f;
    for (int c = 0; c < 32; ++c) acc[c] = 0.f;
    const int last = ctx - rows.y + (first + n_rows - 1) / G, p0 = ctx - rows.y + first / G;  // positions
    const int low = a.window ? max(0, p0 - a.window + 1) : 0;
    for (int page = 0; page * PAGE <= last; ++page) {
        if (page * PAGE >= a.sinks && (page + 1) * PAGE <= low) continue;
        const int id = __ldg(a.block_table + (size_t)b * a.max_pages + page);
        const bool ok = id >= 0 && (int64_t)id < a.num_pages;
        if (!ok && tid == 0) atomicOr(a.error, ERR_BAD_PAGE);
        if (!ok) continue;
        __syncthreads();
        const uint8_t* tile = a.cache + ((size_t)id * a.H_kv + h) * INT4_TILE;
        for (int x = tid; x < PAGE * D; x += 128) {
            const int s = x / D, ch = x % D, g = ch / 32, kt = ch % 32 / 8, ki = ch % 8, vr = ch % 32 / 4, vi = ch % 4;
            const int kc = tile[O4_KC + 64 * s + 16 * kt + 4 * g + ki / 2] >> (4 * (ki & 1)) & 15;
            const int vc = tile[O4_VC + 128 * (s / 2) + 16 * vr + 4 * g + 2 * (s & 1) + vi / 2] >> (4 * (vi & 1)) & 15;
            auto half_at = [&](int at) { return __half2float(*reinterpret_cast<const __half*>(tile + at)); };
            const bool there = page * PAGE + s < ctx;
            K[s][ch] = there ? fmaf((float)kc, half_at(O4_KM + 16 * s + 2 * g), half_at(O4_KM + 16 * s + 8 + 2 * g)) : 0.f;
            V[s][ch] = there ? fmaf((float)vc, half_at(O4_VS + int4_vmeta_off(s, g)), half_at(O4_VM + int4_vmeta_off(s, g))) : 0.f;
        }
        __syncthreads();
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < D; ++c)
            for (int e = 0; e < 4; ++e) x[e] = fmaf(qs[row][c], K[4 * part + e][c], x[e]);
        float top = m;
        for (int e = 0; e < 4; ++e) {
            const int t = page * PAGE + 4 * part + e;
            if (!(t <= pos && (!a.window || t > pos - a.window || t < a.sinks))) x[e] = -CUDART_INF_F;
            top = fmaxf(top, x[e]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float c0 = m == -CUDART_INF_F ? 0.f : exp2f(m - top);
        l *= c0;
        for (int c = 0; c < 32; ++c) acc[c] *= c0;
        m = top;
        float p[4];
        for (int e = 0; e < 4; ++e) {
            p[e] = x[e] == -CUDART_INF_F ? 0.f : exp2f(x[e] - m);
            l += p[e];
        }
        for (int s = 0; s < PAGE; ++s) {
            const float w = __shfl_sync(0xffffffffu, p[s & 3], (tid & 28) | (s >> 2));
            if (w == 0.f) continue;
            for (int c = 0; c < 32; ++c) acc[c] = fmaf(w, V[s][32 * part + c], acc[c]);
        }
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    __syncthreads();
    for (int c = 0; c < 32; ++c) qs[row][32 * part + c] = acc[c] * inv;
    __syncthreads();
    if (!live) return;
    __nv_bfloat16* out = a.out + ((size_t)(rows.x + tok) * a.H_q + head) * D;
    for (int i = 32 * part; i < 32 * part + 32; ++i) {
        float x = 0.f;
        for (int c = 0; c < D; ++c) x = fmaf(qs[row][c], __ldg(a.Rv + ((size_t)h * D + i) * D + c), x);
        out[i] = __float2bfloat16_rn(x);
    }
}

}  // namespace kvq

using namespace kvq;

// What the sizes are refused for (null: nothing).
static const char* chunk_refusal(int n_tok, int B, int H_q, int H_kv, kvq_status& st) {
    st = KVQ_ERR_INVALID_ARG;
    if (n_tok < 0 || B <= 0 || H_kv <= 0 || H_q <= 0 || H_q % H_kv) return "sizes";
    st = KVQ_ERR_UNSUPPORTED;
    if (H_q / H_kv > 64) return "GQA group above 64";
    if (B > 65535 || H_kv > 65535) return "B or H_kv above 65535";
    if ((int64_t)n_tok * H_q > (int64_t(1) << 30)) return "n_tok * H_q above 2^30";
    st = KVQ_OK;
    return nullptr;
}

extern "C" size_t kvq_chunk_workspace_bytes(int n_tok, int B, int H_q, int H_kv) {
    kvq_status st;
    return chunk_refusal(n_tok, B, H_q, H_kv, st) ? 0 : (size_t)WS_HEADER;
}

extern "C" kvq_status kvq_chunk_attn_int4(const void* q, int n_tok, const int32_t* q_start, int B, int H_q, int H_kv, int d,
                                          const void* cache, int64_t num_pages, const int32_t* block_table,
                                          int max_pages_per_seq, const int32_t* context_lens, const float* R_k,
                                          const float* R_v, float scale, int window, int sinks, void* out,
                                          void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "kvq_chunk_attn_int4";
    if (d != D) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: d=%d (only 128)", fn, d);
    kvq_status st;
    if (const char* why = chunk_refusal(n_tok, B, H_q, H_kv, st))
        return kvq_set_error(st, "%s: %s (n_tok=%d B=%d H_q=%d H_kv=%d)", fn, why, n_tok, B, H_q, H_kv);
    if (num_pages <= 0 || max_pages_per_seq <= 0 || window < 0 || sinks < 0)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: num_pages=%lld max_pages=%d window=%d sinks=%d", fn, (long long)num_pages,
                             max_pages_per_seq, window, sinks);
    if (max_pages_per_seq >= (1 << 27)) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: max_pages_per_seq not below 2^27", fn);
    if (num_pages > (int64_t(1) << 32) / H_kv) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: num_pages * H_kv above 2^32", fn);
    if (n_tok == 0) return KVQ_OK;
    if (!q || !q_start || !cache || !block_table || !context_lens || !R_k || !R_v || !out || !workspace)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void* p : {q, cache, (const void*)R_k, (const void*)R_v, (const void*)out, (const void*)workspace})
        if (reinterpret_cast<uintptr_t>(p) % 16)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: q, cache, R_k, R_v, out and workspace need 16-byte alignment", fn);
    if (workspace_bytes < kvq_chunk_workspace_bytes(n_tok, B, H_q, H_kv))
        return kvq_set_error(KVQ_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, workspace_bytes,
                             kvq_chunk_workspace_bytes(n_tok, B, H_q, H_kv));
    ChunkArgs a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.n_tok = n_tok;
    a.q_start = q_start;
    a.B = B;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.G = H_q / H_kv;
    a.cache = static_cast<const uint8_t*>(cache);
    a.num_pages = num_pages;
    a.block_table = block_table;
    a.max_pages = max_pages_per_seq;
    a.context_lens = context_lens;
    a.Rk = R_k;
    a.Rv = R_v;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.window = window;
    a.sinks = window ? sinks : 0;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.error = static_cast<uint32_t*>(workspace);
    const int64_t blocks = ((int64_t)n_tok * a.G + CH_ROWS - 1) / CH_ROWS + B;
    return kvq_check_cuda(launch_pdl(chunk_int4_kernel, dim3((unsigned)blocks, H_kv), dim3(128), 0, static_cast<cudaStream_t>(stream), a),
                          "kvq_chunk_attn_int4 launch");
}
