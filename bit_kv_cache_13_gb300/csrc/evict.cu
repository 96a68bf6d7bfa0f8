// Eviction from the INT4 cache by accumulated attention weight: the selection
// of the tokens each (sequence, KV head) keeps, and the move of the kept
// tokens into other pages.
#include <mutex>

#include "int4_common.cuh"

namespace kvq {

constexpr int SEL_THREADS = 1024, SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_BINS = 2048;                       // bins of a digit (11, 11 and 10 bits)
constexpr int SEL_KEYS = 48 * 1024;                  // keys a CTA holds in shared memory

// Order-preserving key of a weight: larger weight, larger key; -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -CUDART_INF_F;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct __align__(16) SelectSmem {
    int hist[3][SEL_BINS];
    int warp_sum[SEL_WARPS], warp_gt[SEL_WARPS], warp_eq[SEL_WARPS];
    int total_gt, total_eq, digit, above;
};
static_assert(sizeof(SelectSmem) % 16 == 0, "the keys behind it are read sixteen bytes at a time");

// The same shared variable of CTA `rank` of the cluster.
__device__ __forceinline__ int cluster_load(const int* p, int rank) {
    uint32_t addr;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int4 cluster_load4(const int* p, int rank) {
    uint32_t addr;
    int4 v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A cluster of CS CTAs per (sequence, KV head), each with a contiguous run of the
// tokens; candidates are the tokens [sinks, n - recent).  Radix selection of the
// k-th largest key in three digits: a CTA counts its keys in shared memory, the
// cluster's counts are added by reading them from one another's shared memory, and
// the row is read from global memory once (its keys stay in shared memory, up to
// SEL_KEYS per CTA).  Then the kept indices are written in order: every warp counts
// what it keeps of its run, a prefix sum over warps and CTAs gives it its place.
// A lane takes four neighbouring keys at a time.  A row of 128K is bound by these
// steps' latencies (eight rows 23.5 us: a digit 4.5 us, half of it the cluster's barrier
// and reads; counting and writing the kept 8): one CTA per row took 300 us, and reading
// the clusters' counts a word at a time 5 us a digit.
template <int CS>
__global__ void __launch_bounds__(SEL_THREADS)
evict_select_kernel(const float* __restrict__ weights, int64_t stride, int H_kv, int max_tokens,
                    const int32_t* __restrict__ context_lens, int budget, int sinks, int recent,
                    int32_t* __restrict__ keep, int32_t* __restrict__ new_lens, int in_smem) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SelectSmem& sm = *reinterpret_cast<SelectSmem*>(smem_raw);
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(SelectSmem));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CS > 1 ? blockIdx.x % CS : 0, h = (int)(blockIdx.x / CS), b = blockIdx.y;
    griddep_wait();
    griddep_launch_dependents();
    const int n = max(0, min(__ldg(context_lens + b), max_tokens));
    int32_t* out = keep + ((size_t)b * H_kv + h) * budget;
    if (h == 0 && rank == 0 && tid == 0) new_lens[b] = min(n, budget);
    if (n <= budget) {  // (uniform over the cluster)
        for (int i = rank * SEL_THREADS + tid; i < budget; i += CS * SEL_THREADS) out[i] = i < n ? i : -1;
        return;
    }
    const float* w = weights + ((size_t)b * H_kv + h) * stride;
    const int c0 = sinks, c1 = n - recent;  // 0 <= budget - sinks - recent < c1 - c0
    // this CTA's tokens, and each warp's run of them (whole 128s)
    const int per_cta = ((n + CS - 1) / CS + 3) & ~3, t0 = min(n, rank * per_cta), t1 = min(n, t0 + per_cta);
    const int per_warp = ((t1 - t0 + 128 * SEL_WARPS - 1) / (128 * SEL_WARPS)) * 128;
    const int w0 = min(t1, t0 + warp * per_warp), w1 = min(t1, w0 + per_warp), end = w0 + ((w1 - w0 + 127) & ~127);
    for (int i = tid; i < 3 * SEL_BINS; i += SEL_THREADS) (&sm.hist[0][0])[i] = 0;
    __syncthreads();
    // keys i .. i + 3 (0 past the run's end, which no candidate's key is below)
    auto load4 = [&](int i, uint32_t (&key)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) key[q] = i + q < w1 ? weight_key(__ldg(w + i + q)) : 0u;
    };
    auto keys4 = [&](int i, uint32_t (&key)[4]) {
        if (in_smem) {  // (the room behind a run's end holds what the load left there: zeros)
            const uint4 x = *reinterpret_cast<const uint4*>(keys + (i - t0));
            key[0] = x.x;
            key[1] = x.y;
            key[2] = x.z;
            key[3] = x.w;
        } else {
            load4(i, key);
        }
    };
    auto candidate = [&](int i) { return i >= c0 && i < c1 && i < w1; };
    // ---- first digit, while the keys come in
#pragma unroll 2
    for (int i = w0 + 4 * lane; i < end; i += 128) {
        uint32_t key[4];
        load4(i, key);
        if (in_smem && i < w1) *reinterpret_cast<uint4*>(keys + (i - t0)) = make_uint4(key[0], key[1], key[2], key[3]);
        const uint32_t first = __shfl_sync(0xffffffffu, key[0] >> 21, 0);
        const bool whole = candidate(i) && candidate(i + 3);
        if (__all_sync(0xffffffffu, whole && key[0] >> 21 == first && key[1] >> 21 == first && key[2] >> 21 == first && key[3] >> 21 == first)) {
            if (lane == 0) atomicAdd(&sm.hist[0][first], 128);  // (ties: a warp's 128 keys at once)
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (candidate(i + q)) atomicAdd(&sm.hist[0][key[q] >> 21], 1);
        }
    }
    uint32_t prefix = 0;
    int need = budget - sinks - recent;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        if (pass > 0) {
            const int above = pass == 1 ? 21 : 10, shift = pass == 1 ? 10 : 0;
            const uint32_t mask = pass == 1 ? 2047u : 1023u;
#pragma unroll 2
            for (int i = w0 + 4 * lane; i < end; i += 128) {
                uint32_t key[4];
                keys4(min(i, w1 - 1) & ~3, key);
                bool in[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) in[q] = key[q] >> above == prefix && candidate(i + q);
                const uint32_t m = __ballot_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3]);
                if (!m) continue;
                const uint32_t first = __shfl_sync(0xffffffffu, key[0] >> shift & mask, 0);
                bool same = true;
#pragma unroll
                for (int q = 0; q < 4; ++q) same = same && in[q] && (key[q] >> shift & mask) == first;
                if (__all_sync(0xffffffffu, same)) {
                    if (lane == 0) atomicAdd(&sm.hist[pass][first], 128);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (in[q]) atomicAdd(&sm.hist[pass][key[q] >> shift & mask], 1);
                }
            }
        }
        if (CS > 1)
            cluster_barrier();
        else
            __syncthreads();
        // thread t < 512: bins 2047 - 4 t and the three below, so that a prefix sum counts from the top
        const int hi_bin = SEL_BINS - 1 - 4 * tid;
        int4 v = make_int4(0, 0, 0, 0);
        if (tid < SEL_BINS / 4) {
#pragma unroll
            for (int q = 0; q < CS; ++q) {
                const int* p = &sm.hist[pass][hi_bin - 3];
                const int4 x = CS > 1 ? cluster_load4(p, q) : *reinterpret_cast<const int4*>(p);
                v = make_int4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
            }
        }
        const int sum = v.x + v.y + v.z + v.w;
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += z;
        }
        if (lane == 31) sm.warp_sum[warp] = inc;
        __syncthreads();
        int before = inc - sum, lower = lane < warp ? sm.warp_sum[lane] : 0;
#pragma unroll
        for (int o = 16; o; o >>= 1) lower += __shfl_xor_sync(0xffffffffu, lower, o);
        before += lower;  // keys in higher bins than this thread's
        // the digit: the highest bin with need or more keys from the top down to it (for
        // need = 0, the top: nothing lies above it, and nothing equal to it is taken)
        if (need > before && need <= before + sum) {
            const int c[4] = {v.w, v.z, v.y, v.x};
            int q = 0;
            while (before + c[q] < need) before += c[q++];
            sm.digit = hi_bin - q;
            sm.above = before;
        } else if (need == 0 && tid == 0) {
            sm.digit = pass == 2 ? 1023 : SEL_BINS - 1;
            sm.above = 0;
        }
        __syncthreads();
        prefix = pass == 2 ? prefix << 10 | (uint32_t)sm.digit : prefix << 11 | (uint32_t)sm.digit;
        need -= sm.above;
        __syncthreads();  // (the next pass writes digit, above and warp_sum)
    }
    // ---- kept: the protected, keys above `prefix`, and the first `need` equal to it
    auto look = [&](int i, uint32_t& gt, uint32_t& eq) {  // bits of keys i .. i + 3; gt: kept whatever the ties
        uint32_t key[4];
        keys4(min(i, w1 - 1) & ~3, key);
        gt = eq = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bool cand = candidate(i + q);
            gt |= (uint32_t)(i + q < w1 && (!cand || key[q] > prefix)) << q;
            eq |= (uint32_t)(cand && key[q] == prefix) << q;
        }
    };
    int n_gt = 0, n_eq = 0;
    for (int i = w0 + 4 * lane; i < end; i += 128) {
        uint32_t gt, eq;
        look(i, gt, eq);
        n_gt += __popc(gt);
        n_eq += __popc(eq);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        n_gt += __shfl_xor_sync(0xffffffffu, n_gt, o);
        n_eq += __shfl_xor_sync(0xffffffffu, n_eq, o);
    }
    if (lane == 0) {
        sm.warp_gt[warp] = n_gt;
        sm.warp_eq[warp] = n_eq;
    }
    __syncthreads();
    int g = sm.warp_gt[lane], e = sm.warp_eq[lane], g_before = lane < warp ? g : 0, e_before = lane < warp ? e : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        g += __shfl_xor_sync(0xffffffffu, g, o);
        e += __shfl_xor_sync(0xffffffffu, e, o);
        g_before += __shfl_xor_sync(0xffffffffu, g_before, o);
        e_before += __shfl_xor_sync(0xffffffffu, e_before, o);
    }
    if (CS > 1) {
        if (tid == 0) {
            sm.total_gt = g;
            sm.total_eq = e;
        }
        cluster_barrier();
        for (int q = 0; q < rank; ++q) {
            g_before += cluster_load(&sm.total_gt, q);
            e_before += cluster_load(&sm.total_eq, q);
        }
    }
    const uint32_t below = (1u << lane) - 1;
    for (int i = w0 + 4 * lane; i < end; i += 128) {
        uint32_t gt, eq;
        look(i, gt, eq);
        // what the lanes below keep and tie, and the warp
        int g_low = 0, e_low = 0, g_all = 0, e_all = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t m = __ballot_sync(0xffffffffu, gt >> q & 1);
            g_low += __popc(m & below);
            g_all += __popc(m);
        }
        if (__any_sync(0xffffffffu, eq)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t m = __ballot_sync(0xffffffffu, eq >> q & 1);
                e_low += __popc(m & below);
                e_all += __popc(m);
            }
        }
        int g_at = g_before + g_low, e_at = e_before + e_low;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bool is_gt = gt >> q & 1, is_eq = eq >> q & 1;
            const int at = g_at + min(e_at, need);
            if ((is_gt || (is_eq && e_at < need)) && at < budget) out[at] = i + q;
            g_at += is_gt;
            e_at += is_eq;
        }
        g_before += g_all;
        e_before += e_all;
    }
    if (CS > 1) cluster_barrier();  // (shared memory is read from the other CTAs until here)
}

// One warp per (destination page, KV head).  The keys' codes and meta are
// token-major (five 16-byte pieces a token); the values' are two tokens to a
// word, so the two sources of a slot pair are merged half by half.  Bound by its chain
// of three dependent loads (index, page, bytes), so everything of a page is asked for
// before any of it is written: eight heads to 8K tokens 4 us, 21 MB in and out of L2 or
// DRAM; to 2048 in eight sequences 26 us when each piece was written as it came, 19.4 so.
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
    // ---- everything is asked for before anything is written
    uint4 kp[3];           // keys: piece c % 5 (four of codes, one of meta) of token c / 5
    uint16_t va[8], vb[8]; // value codes: word `lane` of each slot pair, its two sources' halves
    uint16_t ma[2], mb[2]; // value meta: word x % 8 (four of scales, four of mins) of pair x / 8
    auto half = [&](int tok, int base, int stride) {  // the source half of a token's word
        const int64_t st = __shfl_sync(0xffffffffu, stile, tok);
        const int ss = __shfl_sync(0xffffffffu, sslot, tok);
        return okm >> tok & 1 ? __ldg(reinterpret_cast<const uint16_t*>(cache + st + base + stride * (ss >> 1) + 2 * (ss & 1)))
                              : (uint16_t)0;
    };
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        const int c = 32 * x + lane, tok = min(c / 5, 15), piece = c % 5;
        const int64_t st = __shfl_sync(0xffffffffu, stile, tok);
        const int ss = __shfl_sync(0xffffffffu, sslot, tok);
        kp[x] = make_uint4(0u, 0u, 0u, 0u);
        if (c < 80 && (okm >> tok & 1))
            kp[x] = __ldg(reinterpret_cast<const uint4*>(cache + st + (piece < 4 ? O4_KC + 64 * ss + 16 * piece : O4_KM + 16 * ss)));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        va[j] = half(2 * j, O4_VC + 4 * lane, 128);
        vb[j] = half(2 * j + 1, O4_VC + 4 * lane, 128);
    }
    const int mbase = (lane & 7) < 4 ? O4_VS + 4 * (lane & 3) : O4_VM + 4 * (lane & 3);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int j = 4 * x + (lane >> 3);
        ma[x] = half(2 * j, mbase, 16);
        mb[x] = half(2 * j + 1, mbase, 16);
    }
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        const int c = 32 * x + lane, tok = min(c / 5, 15), piece = c % 5;
        if (c < 80 && (okm >> tok & 1))
            *reinterpret_cast<uint4*>(dt + (piece < 4 ? O4_KC + 64 * tok + 16 * piece : O4_KM + 16 * tok)) = kp[x];
    }
    auto put = [&](int j, int at, uint16_t x, uint16_t y) {  // a slot pair's word, or the half that is there
        const uint32_t two = okm >> (2 * j) & 3;
        if (two == 3)
            *reinterpret_cast<uint32_t*>(dt + at) = (uint32_t)x | (uint32_t)y << 16;
        else if (two == 1)
            *reinterpret_cast<uint16_t*>(dt + at) = x;
        else if (two == 2)
            *reinterpret_cast<uint16_t*>(dt + at + 2) = y;
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) put(j, O4_VC + 128 * j + 4 * lane, va[j], vb[j]);
#pragma unroll
    for (int x = 0; x < 2; ++x) put(4 * x + (lane >> 3), mbase + 16 * (4 * x + (lane >> 3)), ma[x], mb[x]);
}

}  // namespace kvq

using namespace kvq;

static bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

// The shared memory opt-in, once per kernel and device.
static kvq_status select_smem_once(const void* fn, int which) {
    static std::mutex mu;
    static bool done[64][4] = {};
    int dev = 0;
    kvq_status st = kvq_check_cuda(cudaGetDevice(&dev), "kvq_evict_select: cudaGetDevice");
    if (st != KVQ_OK) return st;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && done[dev][which]) return KVQ_OK;
    st = kvq_check_cuda(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(sizeof(SelectSmem) + SEL_KEYS * 4)),
                        "kvq_evict_select smem attribute");
    if (st == KVQ_OK && dev >= 0 && dev < 64) done[dev][which] = true;
    return st;
}

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
    if (max_tokens > (1 << 30)) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "kvq_evict_select: max_tokens %d above 2^30", max_tokens);
    if (weights_stride < max_tokens)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_evict_select: weights_stride %lld below max_tokens %d",
                             (long long)weights_stride, max_tokens);
    if (!weights || !context_lens || !keep || !new_lens)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_evict_select: null pointer");
    // What is written while other CTAs still read: a late reader of an overwritten length would
    // keep other tokens, and threads that disagree on it would part before a barrier.
    const int64_t rows = (int64_t)B * H_kv;
    const size_t lens_bytes = (size_t)B * 4, keep_bytes = (size_t)rows * budget * 4;
    const size_t weights_bytes = ((size_t)(rows - 1) * weights_stride + max_tokens) * 4;
    if (overlap(new_lens, lens_bytes, context_lens, lens_bytes) || overlap(new_lens, lens_bytes, weights, weights_bytes) ||
        overlap(keep, keep_bytes, context_lens, lens_bytes) || overlap(keep, keep_bytes, weights, weights_bytes) ||
        overlap(keep, keep_bytes, new_lens, lens_bytes))
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_evict_select: keep and new_lens must not overlap another argument");
    // CTAs per row: up to eight (a cluster) while they find an SM each and 2048 tokens or more
    const int nsm = kvq_device_sm_count();
    int cs = 1;
    while (cs < 8 && rows * cs * 2 <= nsm && max_tokens / (cs * 2) >= 2048) cs *= 2;
    const int64_t seg = (((int64_t)max_tokens + cs - 1) / cs + 3) & ~int64_t(3);
    const int in_smem = seg <= SEL_KEYS;
    const size_t smem = sizeof(SelectSmem) + (in_smem ? (size_t)seg * 4 : 0);
    using Kern = decltype(&evict_select_kernel<1>);
    const Kern kern = cs == 8 ? evict_select_kernel<8> : cs == 4 ? evict_select_kernel<4> : cs == 2 ? evict_select_kernel<2> : evict_select_kernel<1>;
    const kvq_status sa = select_smem_once((const void*)kern, cs == 8 ? 3 : cs >> 1);
    if (sa != KVQ_OK) return sa;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(H_kv * cs, B);
    cfg.blockDim = dim3(SEL_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    return kvq_check_cuda(cudaLaunchKernelEx(&cfg, kern, weights, weights_stride, H_kv, max_tokens, context_lens, budget, sinks,
                                             recent, keep, new_lens, in_smem),
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
        // rows of the one between rows of the other are fine, a common float is read by one CTA and written by another
        const size_t last = (size_t)B * H_kv - 1, from = (size_t)max_pages_per_seq * PAGE, to = (size_t)dst_max_pages * PAGE;
        if (overlap(weights, (last * weights_stride + from) * 4, weights_out, (last * weights_out_stride + to) * 4)) {
            const int64_t floats = weights_out - weights, at = ((floats % weights_stride) + weights_stride) % weights_stride;
            if (last == 0 || weights_stride != weights_out_stride || at < (int64_t)from || at + (int64_t)to > weights_stride)
                return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: weights_out must not overlap weights", fn);
        }
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
