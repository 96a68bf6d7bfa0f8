// Eviction from the INT4 cache by accumulated attention weight: the selection
// of the tokens each (sequence, KV head) keeps, and the move of the kept
// tokens into other pages.
#include "int4_common.cuh"

namespace kvq {

constexpr int SEL_THREADS = 1024;

// Order-preserving key of a weight: larger weight, larger key; -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -CUDART_INF_F;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, KV head).  Candidates are the tokens [sinks, n -
// recent); the k-th largest key is found by a radix search, eight bits a pass
// over the row, and the kept indices are written in order by a running count.
__global__ void __launch_bounds__(SEL_THREADS)
evict_select_kernel(const float* __restrict__ weights, int64_t stride, int H_kv, int max_tokens,
                    const int32_t* __restrict__ context_lens, int budget, int sinks, int recent,
                    int32_t* __restrict__ keep, int32_t* __restrict__ new_lens) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ int hist[256], warp_eq[32], warp_kept[32];
    __shared__ uint32_t s_digit;
    __shared__ int s_above;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = max(0, min(__ldg(context_lens + b), max_tokens));
    int32_t* out = keep + ((size_t)b * H_kv + h) * budget;
    if (h == 0 && tid == 0) new_lens[b] = min(n, budget);
    if (n <= budget) {
        for (int i = tid; i < budget; i += SEL_THREADS) out[i] = i < n ? i : -1;
        return;
    }
    const float* w = weights + ((size_t)b * H_kv + h) * stride;
    const int c0 = sinks, c1 = n - recent, k = budget - sinks - recent;  // 0 <= k < c1 - c0
    uint32_t prefix = 0;
    int need = k;
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i = c0 + tid; i < c1; i += SEL_THREADS) {
            const uint32_t key = weight_key(__ldg(w + i));
            if (pass == 0 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int above = 0, dgt = 255;
            for (; dgt > 0 && above + hist[dgt] < need; --dgt) above += hist[dgt];
            s_digit = (uint32_t)dgt;
            s_above = above;
        }
        __syncthreads();
        prefix = (prefix << 8) | s_digit;
        need -= s_above;
        __syncthreads();
    }
    // kept candidates: keys above `prefix`, and the first `need` equal to it
    int base_kept = 0, base_eq = 0;
    for (int i0 = 0; i0 < n; i0 += SEL_THREADS) {
        const int i = i0 + tid;
        const bool cand = i >= c0 && i < c1, prot = i < n && !cand;
        const uint32_t key = cand ? weight_key(__ldg(w + i)) : 0u;
        const bool eq = cand && key == prefix;
        const uint32_t meq = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) warp_eq[warp] = __popc(meq);
        __syncthreads();
        int eq_before = base_eq + __popc(meq & ((1u << lane) - 1));
        int eq_all = 0;
        for (int x = 0; x < 32; ++x) {
            if (x < warp) eq_before += warp_eq[x];
            eq_all += warp_eq[x];
        }
        const bool kept = prot || (cand && key > prefix) || (eq && eq_before < need);
        const uint32_t mk = __ballot_sync(0xffffffffu, kept);
        if (lane == 0) warp_kept[warp] = __popc(mk);
        __syncthreads();
        int at = base_kept + __popc(mk & ((1u << lane) - 1)), all = 0;
        for (int x = 0; x < 32; ++x) {
            if (x < warp) at += warp_kept[x];
            all += warp_kept[x];
        }
        if (kept && at < budget) out[at] = i;
        base_kept += all;
        base_eq += eq_all;
        __syncthreads();
    }
}

// One warp per (destination page, KV head).  The keys' codes and meta are
// token-major (five 16-byte pieces a token); the values' are two tokens to a
// word, so the two sources of a slot pair are merged half by half.
constexpr int GATHER_WARPS = 4;

__global__ void __launch_bounds__(GATHER_WARPS * 32)
evict_gather_int4_kernel(const uint8_t* cache, int64_t num_pages, const int32_t* __restrict__ block_table,
                         int max_pages, const int32_t* __restrict__ keep, int budget,
                         const int32_t* __restrict__ new_lens, int H_kv, uint8_t* dst,
                         int64_t dst_num_pages, const int32_t* __restrict__ dst_block_table, int dst_max_pages,
                         const float* __restrict__ weights, int64_t wstride, float* __restrict__ weights_out,
                         int64_t wostride, int32_t* __restrict__ err_count) {
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int p = blockIdx.x * GATHER_WARPS + warp, h = blockIdx.y, b = blockIdx.z;
    if (p >= dst_max_pages) return;
    const size_t unit = (size_t)b * H_kv + h;
    const int nl = max(0, min(__ldg(new_lens + b), budget));
    // lane i < 16: destination token 16 p + i and its source
    const int i = p * PAGE + (lane & 15);
    const bool there = i < nl;
    const int src = there ? __ldg(keep + unit * budget + i) : -1;
    const int did = there ? __ldg(dst_block_table + (size_t)b * dst_max_pages + p) : -1;
    const bool idx_ok = there && src >= 0 && src < max_pages * PAGE;
    const int sid = idx_ok ? __ldg(block_table + (size_t)b * max_pages + src / PAGE) : -1;
    const bool src_ok = idx_ok && sid >= 0 && (int64_t)sid < num_pages;
    const bool dst_ok = did >= 0 && (int64_t)did < dst_num_pages;
    const bool ok = src_ok && dst_ok;
    if (weights && lane < 16)
        weights_out[unit * wostride + i] = src_ok ? __ldg(weights + unit * wstride + src) : 0.f;
    const uint32_t bad = __ballot_sync(0xffffffffu, there && !ok && lane < 16);
    if (bad && lane == 0 && err_count) atomicAdd(err_count, __popc(bad));
    const uint32_t okm = __ballot_sync(0xffffffffu, ok) & 0xffffu;
    if (!okm) return;
    const int64_t stile = ((int64_t)sid * H_kv + h) * INT4_TILE;
    const int sslot = src & (PAGE - 1);
    uint8_t* dt = dst + ((size_t)__shfl_sync(0xffffffffu, did, 0) * H_kv + h) * INT4_TILE;  // (token 0 is there if any is)
#pragma unroll
    for (int c0 = 0; c0 < 96; c0 += 32) {
        const int c = c0 + lane, tok = min(c / 5, 15), piece = c % 5;
        const int64_t st = __shfl_sync(0xffffffffu, stile, tok);
        const int ss = __shfl_sync(0xffffffffu, sslot, tok);
        if (c < 80 && (okm >> tok & 1)) {
            const int so = piece < 4 ? O4_KC + 64 * ss + 16 * piece : O4_KM + 16 * ss;
            const int to = piece < 4 ? O4_KC + 64 * tok + 16 * piece : O4_KM + 16 * tok;
            *reinterpret_cast<uint4*>(dt + to) = *reinterpret_cast<const uint4*>(cache + st + so);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t sa = __shfl_sync(0xffffffffu, stile, 2 * j), sb = __shfl_sync(0xffffffffu, stile, 2 * j + 1);
        const int la = __shfl_sync(0xffffffffu, sslot, 2 * j), lb = __shfl_sync(0xffffffffu, sslot, 2 * j + 1);
        const bool oa = okm >> (2 * j) & 1, ob = okm >> (2 * j + 1) & 1;
        // 32 words of codes, then 4 scale and 4 min words
        for (int w = lane; w < 40; w += 32) {
            const int base = w < 32 ? O4_VC + 4 * w : (w < 36 ? O4_VS : O4_VM) + 4 * (w & 3), stride = w < 32 ? 128 : 16;
            uint16_t* d16 = reinterpret_cast<uint16_t*>(dt + base + stride * j);
            if (oa) d16[0] = *reinterpret_cast<const uint16_t*>(cache + sa + base + stride * (la >> 1) + 2 * (la & 1));
            if (ob) d16[1] = *reinterpret_cast<const uint16_t*>(cache + sb + base + stride * (lb >> 1) + 2 * (lb & 1));
        }
    }
}

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_evict_select(const float* weights, int64_t weights_stride, int B, int H_kv, int max_tokens,
                                       const int32_t* context_lens, int budget, int sinks, int recent, int32_t* keep,
                                       int32_t* new_lens, void* stream) {
    if (B <= 0 || H_kv <= 0 || max_tokens <= 0 || budget <= 0 || sinks < 0 || recent < 0)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_evict_select: B=%d H_kv=%d max_tokens=%d budget=%d sinks=%d recent=%d",
                             B, H_kv, max_tokens, budget, sinks, recent);
    if ((int64_t)sinks + recent > budget)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_evict_select: sinks %d + recent %d above the budget %d", sinks, recent,
                             budget);
    if (B > 65535 || H_kv > 65535) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "kvq_evict_select: B or H_kv above 65535");
    if (weights_stride < max_tokens)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_evict_select: weights_stride %lld below max_tokens %d",
                             (long long)weights_stride, max_tokens);
    if (!weights || !context_lens || !keep || !new_lens)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_evict_select: null pointer");
    return kvq_check_cuda(launch_pdl(evict_select_kernel, dim3(H_kv, B), dim3(SEL_THREADS), 0,
                                     static_cast<cudaStream_t>(stream), weights, weights_stride, H_kv, max_tokens,
                                     context_lens, budget, sinks, recent, keep, new_lens),
                          "kvq_evict_select launch");
}

extern "C" kvq_status kvq_evict_gather_int4(const void* cache, int64_t num_pages, const int32_t* block_table,
                                            int max_pages_per_seq, const int32_t* keep, int budget,
                                            const int32_t* new_lens, int B, int H_kv, int d, void* dst_cache,
                                            int64_t dst_num_pages, const int32_t* dst_block_table, int dst_max_pages,
                                            const float* weights, int64_t weights_stride, float* weights_out,
                                            int64_t weights_out_stride, int32_t* err_count, void* stream) {
    const char* fn = "kvq_evict_gather_int4";
    if (d != D) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: d=%d (only 128)", fn, d);
    if (B <= 0 || H_kv <= 0 || num_pages <= 0 || max_pages_per_seq <= 0 || budget <= 0 || dst_num_pages <= 0 ||
        dst_max_pages <= 0)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: B=%d H_kv=%d num_pages=%lld max_pages=%d budget=%d dst_num_pages=%lld "
                             "dst_max_pages=%d", fn, B, H_kv, (long long)num_pages, max_pages_per_seq, budget,
                             (long long)dst_num_pages, dst_max_pages);
    if (B > 65535 || H_kv > 65535) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: B or H_kv above 65535", fn);
    if (max_pages_per_seq >= (1 << 27) || dst_max_pages >= (1 << 27))
        return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: pages per sequence not below 2^27", fn);
    if ((int64_t)dst_max_pages * PAGE < budget)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: %d destination pages hold fewer than %d tokens", fn, dst_max_pages,
                             budget);
    if (!cache || !block_table || !keep || !new_lens || !dst_cache || !dst_block_table || (weights && !weights_out))
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(dst_cache) % 16)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: caches need 16-byte alignment", fn);
    if (weights) {
        if (weights_stride < (int64_t)max_pages_per_seq * PAGE || weights_out_stride < (int64_t)dst_max_pages * PAGE)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: weights strides %lld, %lld below 16 * pages per sequence", fn,
                                 (long long)weights_stride, (long long)weights_out_stride);
        if (weights == weights_out) return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: weights_out is weights", fn);
    }
    // pages past the budget only have weights to clear
    const int pages = weights ? dst_max_pages : (budget + PAGE - 1) / PAGE;
    return kvq_check_cuda(launch_pdl(evict_gather_int4_kernel, dim3((pages + GATHER_WARPS - 1) / GATHER_WARPS, H_kv, B),
                                     dim3(GATHER_WARPS * 32), 0, static_cast<cudaStream_t>(stream),
                                     static_cast<const uint8_t*>(cache), num_pages, block_table, max_pages_per_seq, keep,
                                     budget, new_lens, H_kv, static_cast<uint8_t*>(dst_cache), dst_num_pages,
                                     dst_block_table, dst_max_pages, weights, weights_stride, weights_out,
                                     weights_out_stride, err_count),
                          "kvq_evict_gather_int4 launch");
}
