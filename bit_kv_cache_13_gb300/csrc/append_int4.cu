// Quantise-on-append and read-back of the rotated INT4 KV cache.
//
// z = (k - mu) R_k, w = v R_v, then 16 levels per group of 32 rotated channels
// with an fp16 scale and min.  Codes, scales and mins are those of the exact
// rotated vectors, whichever kernel writes them: each kernel forms the rotated
// values to within a bound, and where a rounding or a threshold lies within that
// bound of a value (a few groups in a hundred) it forms the value exactly.
#include <cstddef>
#include <mutex>
#include <type_traits>

#include "int4_common.cuh"

namespace kvq {

// Writes code word w (8 codes: channels 32 g + 8 t + i of nibble i) of one token.
__device__ __forceinline__ void store_word(uint8_t* tile, int side, int s, int g, int t, uint32_t w) {
    if (!side) {
        *reinterpret_cast<uint32_t*>(tile + O4_KC + 64 * s + 16 * t + 4 * g) = w;
    } else {
        uint8_t* p = tile + O4_VC + 128 * (s >> 1) + 32 * t + 4 * g + 2 * (s & 1);
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)w;
        *reinterpret_cast<uint16_t*>(p + 16) = (uint16_t)(w >> 16);
    }
}

__device__ __forceinline__ void store_meta(uint8_t* tile, int side, int s, int g, __half sh, __half mh) {
    if (!side) {
        *reinterpret_cast<__half*>(tile + O4_KM + 16 * s + 2 * g) = sh;
        *reinterpret_cast<__half*>(tile + O4_KM + 16 * s + 8 + 2 * g) = mh;
    } else {
        *reinterpret_cast<__half*>(tile + O4_VS + int4_vmeta_off(s, g)) = sh;
        *reinterpret_cast<__half*>(tile + O4_VM + int4_vmeta_off(s, g)) = mh;
    }
}

// ------------------------------------------------------------ a few tokens
//
// One CTA of 512 threads per (token, KV head, side): thread (channel, quarter)
// sums 32 products in an unevaluated pair of fp32 values, so the rotated values are
// exact to about 46 bits and no second look is taken.  Bound by its chain of
// latencies: one row of R_k per thread and quarter in flight.

__global__ void __launch_bounds__(512)
append_int4_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v, int n_tok, int H_kv,
                   const int32_t* __restrict__ slot_mapping, const float* __restrict__ mu,
                   const float* __restrict__ Rk, const float* __restrict__ Rv, uint8_t* __restrict__ cache,
                   int64_t num_pages, int32_t* __restrict__ err_count, float clip) {
    __shared__ float xs[D], xl[D], n2s[4];
    __shared__ Dd part[4][D];
    const int t = blockIdx.x, h = blockIdx.y, side = blockIdx.z, tid = threadIdx.x;
    const int j = tid & (D - 1), quarter = tid >> 7, lane = tid & 31, g = (tid >> 5) & 3;
    const float* R = (side ? Rv : Rk) + (size_t)h * D * D + (size_t)32 * quarter * D + j;
    prefetch_l2(R - j + (size_t)(j >> 2) * D + 32 * (j & 3));  // the quarter's 32 rows, four lines each
    griddep_wait();
    griddep_launch_dependents();
    const int slot = __ldg(slot_mapping + t);
    float rr[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) rr[i] = __ldg(R + (size_t)i * D);
    if (slot < 0 || (int64_t)slot >= num_pages * PAGE) {
        if (slot != -1 && tid == 0 && h == 0 && side == 0 && err_count) atomicAdd(err_count, 1);
        return;
    }
    if (quarter == 0) {
        const size_t row = ((size_t)t * H_kv + h) * D + j;
        const float x = __bfloat162float(side ? v[row] : k[row]);
        const float m = side ? 0.f : __ldg(mu + (size_t)h * D + j);
        float hi, lo;
        two_sum(x, -m, hi, lo);  // (not finite: hi is, too, and lo does not matter)
        xs[j] = hi;
        xl[j] = isfinite(hi) ? lo : 0.f;
        float n2 = fmaf(x, x, m * m);
#pragma unroll
        for (int o = 16; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
        if (lane == 0) n2s[g] = n2;
    }
    __syncthreads();
    const bool wild = int4_wild(n2s[0] + n2s[1] + n2s[2] + n2s[3]);  // CTA-uniform
    if (!wild) {
        // four chains, so that their latencies overlap
        Dd acc[4] = {};
#pragma unroll
        for (int i = 0; i < 32; i += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) dd_fma(acc[e], xs[32 * quarter + i + e], xl[32 * quarter + i + e], rr[i + e]);
        dd_add(acc[0], acc[1]);
        dd_add(acc[2], acc[3]);
        dd_add(acc[0], acc[2]);
        part[quarter][j] = acc[0];
    }
    __syncthreads();
    if (quarter) return;
    __half sh, mh;
    int code;
    if (!wild) {
        Dd z = part[0][j], y = part[2][j];
        dd_add(z, part[1][j]);
        dd_add(y, part[3][j]);
        dd_add(z, y);
        z = dd_norm(z);
        Dd mn = z, mx = z;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const Dd a = {__shfl_xor_sync(0xffffffffu, mn.hi, o), __shfl_xor_sync(0xffffffffu, mn.lo, o)};
            const Dd b = {__shfl_xor_sync(0xffffffffu, mx.hi, o), __shfl_xor_sync(0xffffffffu, mx.lo, o)};
            if (dd_less(a, mn)) mn = a;
            if (dd_less(mx, b)) mx = b;
        }
        int4_params(mn, mx, clip, sh, mh);
        const float s = __half2float(sh), m = __half2float(mh);
        // the nearest threshold decides between two codes (past the ends, and for s = 0, the end)
        const float q = s > 0.f ? fmaf(z.hi - m, 1.f / s, -0.5f) : -1.f;
        code = q <= -0.5f ? 0 : q >= INT4_LEVELS - 0.5f ? INT4_LEVELS : int4_code(z, s, m, (int)rintf(q));
    } else {  // all in fp64
        const float* Rw = (side ? Rv : Rk) + (size_t)h * D * D + j;
        double z = 0.0;
        for (int i = 0; i < D; ++i) z = fma((double)xs[i] + (double)xl[i], (double)__ldg(Rw + (size_t)i * D), z);
        double lo = z, hi = z;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (__any_sync(0xffffffffu, !isfinite(z))) lo = hi = CUDART_NAN;
        int4_params(lo, hi, (double)clip, sh, mh);
        code = int4_code(z, sh, mh);
    }
    // the eight codes of a word sit in eight neighbouring lanes
    uint32_t w = (uint32_t)code << (4 * (lane & 7));
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    uint8_t* tile = cache + ((size_t)(slot / PAGE) * H_kv + h) * INT4_TILE;
    if ((lane & 7) == 0) store_word(tile, side, slot % PAGE, g, lane >> 3, w);
    if (lane == 0) store_meta(tile, side, slot % PAGE, g, sh, mh);
}

// ------------------------------------------------------------ prefill
//
// The rotation on the tensor cores.  The inputs are bf16 and so exact operands; R
// enters as three bf16 parts (its fp32 value to 2^-25), smallest first, into one
// fp32 accumulator, and the centre is subtracted after the rotation (z = k R - mu R,
// mu R formed once per CTA).  A warp owns one group of 32 rotated channels and keeps
// its part of R in 192 registers; a tile is 16 tokens, whose rows all four warps
// read.  With the columns of the product in the order channel 8 t + 2 i + e = column
// 2 t + e of its eight columns' set i, the accumulators of a lane are the eight codes
// of one word of the key record.
//
// |z - accumulated| <= PF_EPS (|k| + |mu|): the largest error seen was 2^-22.1 of the
// norms (2 10^8 values of three distributions), the bound leaves a factor of four.
// Groups or codes that the bound leaves open (about one group in twenty-five, one
// code in ten thousand) take exact dot products by the whole warp, in pairs of fp32
// values: fp64 is 64 times slower than fp32 here, and a first form of these second
// looks in fp64 took most of the kernel's time (32K tokens 1.10 ms).
constexpr int PF_M = 16;                 // tokens of a tile
constexpr float PF_EPS = 0x1p-20f;
constexpr int PF_LIST = 192;             // exact values of a tile (a full one sends its groups the slow way)
constexpr int PF_RT = D + 4, PF_A = D + 8;  // padded rows, in elements

struct __align__(16) PrefillSmem {
    __align__(16) float RT[D][PF_RT];    // R transposed: RT[channel][input]
    __align__(16) __nv_bfloat16 A[2][PF_M][PF_A];
    __align__(16) float mu[D];           // the centre (0 for values)
    __align__(16) float c[D];            // mu R
    __align__(16) uint32_t word[PF_M][4][4];  // the tile's codes [token][t][g]
    __align__(16) __half sc[PF_M][NGROUP];
    __align__(16) __half mn[PF_M][NGROUP];
    __align__(16) Dd found[PF_LIST];     // exact values, of
    uint16_t item[PF_LIST];              // row << 7 | channel
    float eps[PF_M];                     // the bound on the rows' errors; -1: a row for fp64
    int slot[2][PF_M];
    float m2[4], mu2;
    int n_item;
};
static_assert(offsetof(PrefillSmem, RT) % 16 == 0 && offsetof(PrefillSmem, A) % 16 == 0 && offsetof(PrefillSmem, mu) % 16 == 0 &&
                  offsetof(PrefillSmem, c) % 16 == 0 && offsetof(PrefillSmem, word) % 16 == 0 && offsetof(PrefillSmem, sc) % 8 == 0 &&
                  offsetof(PrefillSmem, mn) % 8 == 0 && (PF_RT * 4) % 16 == 0 && (PF_A * 2) % 16 == 0,
              "wide accesses to shared memory are aligned");

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}

// x = p0 + p1 + p2 + (less than 2^-25 of x), bf16 parts
__device__ __forceinline__ float bf16_part(float& x) {
    const float p = __bfloat162float(__float2bfloat16_rn(x));
    x = x - p;  // exact
    return p;
}

__global__ void __launch_bounds__(128, 2)
append_int4_prefill_kernel(const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v, int n_tok, int H_kv,
                           const int32_t* __restrict__ slot_mapping, const float* __restrict__ mu,
                           const float* __restrict__ Rk, const float* __restrict__ Rv, uint8_t* __restrict__ cache,
                           int64_t num_pages, int32_t* __restrict__ err_count, float clip) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    PrefillSmem& sm = *reinterpret_cast<PrefillSmem*>(smem_raw);
    const int h = blockIdx.y, side = blockIdx.z, tid = threadIdx.x, g = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, t = lane & 3;
    const float* R = (side ? Rv : Rk) + (size_t)h * D * D;
    for (int l = tid; l < D * D / 32; l += 128) prefetch_l2(R + 32 * l);
    griddep_wait();
    griddep_launch_dependents();

    const int tiles = (n_tok + PF_M - 1) / PF_M;
    const __nv_bfloat16* src = side ? v : k;
    const int64_t n_slots = num_pages * PAGE;
    auto fetch = [&](int x, int buf) {  // tile x: 256 pieces of 16 bytes, and its slots
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int p = tid + 128 * e, row = p >> 4, col = 8 * (p & 15);
            const int64_t tok = min((int64_t)x * PF_M + row, (int64_t)n_tok - 1);  // (rows past the end repeat the last)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&sm.A[buf][row][col])),
                         "l"(src + ((size_t)tok * H_kv + h) * D + col)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (tid < PF_M) {
            const int64_t tok = (int64_t)x * PF_M + tid;
            int s = tok < n_tok ? __ldg(slot_mapping + tok) : -1;
            if (s != -1 && (s < 0 || (int64_t)s >= n_slots)) {
                if (h == 0 && side == 0 && err_count) atomicAdd(err_count, 1);
                s = -1;
            }
            sm.slot[buf][tid] = s;
        }
    };
    if ((int)blockIdx.x < tiles) fetch(blockIdx.x, 0);
    // R transposed: thread = input row
#pragma unroll 8
    for (int c4 = 0; c4 < D; c4 += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(R + (size_t)tid * D + c4));
        sm.RT[c4][tid] = x.x;
        sm.RT[c4 + 1][tid] = x.y;
        sm.RT[c4 + 2][tid] = x.z;
        sm.RT[c4 + 3][tid] = x.w;
    }
    const float mu_own = side ? 0.f : __ldg(mu + (size_t)h * D + tid);
    sm.mu[tid] = mu_own;
    {
        float m2 = mu_own * mu_own;
#pragma unroll
        for (int o = 16; o; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
        if (lane == 0) sm.m2[g] = m2;
    }
    __syncthreads();
    if (tid == 0) sm.mu2 = (sm.m2[0] + sm.m2[1]) + (sm.m2[2] + sm.m2[3]);
    if (side == 0) {  // mu R: thread = channel
        Dd acc[4] = {};
#pragma unroll 4
        for (int i = 0; i < D; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(&sm.RT[tid][i]);
            dd_fma(acc[0], sm.mu[i], 0.f, x.x);
            dd_fma(acc[1], sm.mu[i + 1], 0.f, x.y);
            dd_fma(acc[2], sm.mu[i + 2], 0.f, x.z);
            dd_fma(acc[3], sm.mu[i + 3], 0.f, x.w);
        }
        dd_add(acc[0], acc[1]);
        dd_add(acc[2], acc[3]);
        dd_add(acc[0], acc[2]);
        sm.c[tid] = acc[0].hi + acc[0].lo;
    } else {
        sm.c[tid] = 0.f;
    }
    // this warp's channels of R as operands: column n of set i is channel 32 g + 8 (n / 2) + 2 i + n % 2
    uint32_t bf[3][4][8][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float2 x = *reinterpret_cast<const float2*>(&sm.RT[32 * g + 8 * (r >> 1) + 2 * i + (r & 1)][16 * ks + 8 * e + 2 * t]);
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const float lo = bf16_part(x.x), hi = bf16_part(x.y);
                    bf[p][i][ks][e] = pack_bf16(lo, hi);
                }
            }

    int buf = 0;
#pragma unroll 1
    for (int x = blockIdx.x; x < tiles; x += gridDim.x, buf ^= 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the tile is there; the last one's words are written out
        {   // norms: 8 threads a row
            const int row = tid >> 3;
            const uint4* p = reinterpret_cast<const uint4*>(&sm.A[buf][row][16 * (tid & 7)]);
            float n2 = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint4 q = p[e];
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float a = __uint_as_float(w[y] << 16), b = __uint_as_float(w[y] & 0xffff0000u);
                    n2 = fmaf(a, a, fmaf(b, b, n2));
                }
            }
            n2 += __shfl_xor_sync(0xffffffffu, n2, 1);
            n2 += __shfl_xor_sync(0xffffffffu, n2, 2);
            n2 += __shfl_xor_sync(0xffffffffu, n2, 4);
            if ((tid & 7) == 0) sm.eps[row] = int4_wild(n2 + sm.mu2) ? -1.f : PF_EPS * (sqrtf(n2) + sqrtf(sm.mu2));
            if (tid == 0) sm.n_item = 0;
        }
        if (x + (int)gridDim.x < tiles) fetch(x + gridDim.x, buf ^ 1);

        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
        const uint32_t a_addr = smem_u32(&sm.A[buf][lane & 15][8 * (lane >> 4)]);
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t a[4];
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                             : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                             : "r"(a_addr + 32 * ks));
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_bf16(acc[i], a, bf[p][i][ks][0], bf[p][i][ks][1]);
            }
        __syncthreads();  // the bounds are there

        // (k - mu) . R[:, ch] (or v . R) of a row: the threads of a group of 2^LOG lanes
        // take four inputs at a time; every lane of the group gets the sum
        auto exact = [&](int row, int ch, auto log) {
            constexpr int LANES = 1 << decltype(log)::value;
            const int q = lane & (LANES - 1);
            Dd s[2] = {};
#pragma unroll
            for (int x = 0; x < 32 / LANES; ++x) {
                const int at = 4 * (LANES * x + q);
                const uint2 raw = *reinterpret_cast<const uint2*>(&sm.A[buf][row][at]);
                const float4 rv = *reinterpret_cast<const float4*>(&sm.RT[ch][at]);
                const float xv[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u),
                                     __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)};
                const float rw[4] = {rv.x, rv.y, rv.z, rv.w};
                if (side) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) dd_fma(s[e & 1], xv[e], 0.f, rw[e]);
                } else {
                    const float4 m4 = *reinterpret_cast<const float4*>(&sm.mu[at]);
                    const float mv[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float hi, lo;
                        two_sum(xv[e], -mv[e], hi, lo);
                        dd_fma(s[e & 1], hi, lo, rw[e]);
                    }
                }
            }
            dd_add(s[0], s[1]);
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1) {
                Dd y;
                y.hi = __shfl_xor_sync(0xffffffffu, s[0].hi, o);
                y.lo = __shfl_xor_sync(0xffffffffu, s[0].lo, o);
                dd_add(s[0], y);
            }
            // (the butterfly adds in another order in each lane: take the group's first)
            s[0].hi = __shfl_sync(0xffffffffu, s[0].hi, lane & ~(LANES - 1));
            s[0].lo = __shfl_sync(0xffffffffu, s[0].lo, lane & ~(LANES - 1));
            return dd_norm(s[0]);
        };
        auto z_of = [&](int i, int e) { return acc[i >> 1][2 * e + (i & 1)]; };
        if (side == 0) {
            const float4 ca = *reinterpret_cast<const float4*>(&sm.c[32 * g + 8 * t]), cb = *reinterpret_cast<const float4*>(&sm.c[32 * g + 8 * t + 4]);
            const float cc[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i >> 1][2 * e + (i & 1)] -= cc[i];
        }
        // ---- each row's parameters; the candidates of open ones go on the CTA's list
        float mn[2], mx[2];
        __half sh[2], mh[2];
        uint32_t cand[2];
        int at[2];
        bool slow[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mn[e] = mx[e] = z_of(0, e);
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                mn[e] = fminf(mn[e], z_of(i, e));
                mx[e] = fmaxf(mx[e], z_of(i, e));
            }
            mn[e] = fminf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mn[e] = fminf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], 2));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
            const float eps = sm.eps[r + 8 * e];
            const bool open = int4_params_near(mn[e], mx[e], clip, eps, sh[e], mh[e]) && eps >= 0.f && sm.slot[buf][r + 8 * e] >= 0;
            cand[e] = 0;
            at[e] = 0;
            slow[e] = false;
            if (__any_sync(0xffffffffu, open)) {
                if (open) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        cand[e] |= (uint32_t)(z_of(i, e) <= mn[e] + 2.f * eps || z_of(i, e) >= mx[e] - 2.f * eps) << i;
                }
                int n = __popc(cand[e]), inc = n, base = 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                if (lane == 31) base = atomicAdd(&sm.n_item, inc);
                base = __shfl_sync(0xffffffffu, base, 31);
                slow[e] = base + __shfl_sync(0xffffffffu, inc, 31) > PF_LIST;  // (warp-uniform)
                at[e] = base + inc - n;
                if (!slow[e]) {
                    int x = at[e];
                    for (uint32_t c = cand[e]; c; c &= c - 1) sm.item[x++] = (uint16_t)((r + 8 * e) << 7 | (32 * g + 8 * t + __ffs(c) - 1));
                } else {
                    for (int x = max(base, 0) + lane; x < PF_LIST; x += 32) sm.item[x] = 0;  // (the list's end stays readable)
                }
            }
        }
        __syncthreads();  // the list is complete
        const int n_item = min(sm.n_item, PF_LIST);
        if (n_item > 0) {
            for (int x0 = 0; x0 < n_item; x0 += 16) {  // eight threads an item
                const int x = x0 + (tid >> 3), it = sm.item[min(x, n_item - 1)];
                const Dd y = exact(it >> 7, it & 127, std::integral_constant<int, 3>());
                if (x < n_item && (lane & 7) == 0) sm.found[x] = y;
            }
            __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = r + 8 * e;
            const bool live = sm.slot[buf][row] >= 0;
            const float eps = sm.eps[row];
            const bool wild = live && eps < 0.f;
            if (__any_sync(0xffffffffu, cand[e] != 0)) {
                // the exact ends of the open groups: every value that could be one was looked at
                Dd lo = {CUDART_INF_F, 0.f}, hi = {-CUDART_INF_F, 0.f};
                if (!slow[e]) {
                    for (int x = 0, n = __popc(cand[e]); x < n; ++x) {
                        const Dd y = sm.found[at[e] + x];
                        if (dd_less(y, lo)) lo = y;
                        if (dd_less(hi, y)) hi = y;
                    }
                } else {  // the list is full: the warp takes its own candidates one by one
                    uint32_t left = cand[e], any;
                    while ((any = __ballot_sync(0xffffffffu, left != 0)) != 0) {
                        const int l = __ffs(any) - 1, i = __ffs(__shfl_sync(0xffffffffu, left, l)) - 1;
                        const Dd y = exact((l >> 2) + 8 * e, 32 * g + 8 * (l & 3) + i, std::integral_constant<int, 5>());
                        if (lane == l) {
                            if (dd_less(y, lo)) lo = y;
                            if (dd_less(hi, y)) hi = y;
                            left &= left - 1;
                        }
                    }
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    const Dd a = {__shfl_xor_sync(0xffffffffu, lo.hi, o), __shfl_xor_sync(0xffffffffu, lo.lo, o)};
                    const Dd b = {__shfl_xor_sync(0xffffffffu, hi.hi, o), __shfl_xor_sync(0xffffffffu, hi.lo, o)};
                    if (dd_less(a, lo)) lo = a;
                    if (dd_less(hi, b)) hi = b;
                }
                if (lo.hi <= hi.hi) int4_params(lo, hi, clip, sh[e], mh[e]);  // (the rows that were not open saw none)
            }
            // ---- codes: the nearest integer to (z - min) / scale within [0, 15], by adding 1.5 2^23;
            // what it leaves of the quotient says how near a threshold is
            const float s = __half2float(sh[e]), m = __half2float(mh[e]), inv = s > 0.f ? 1.f / s : 0.f, off = -m * inv;
            const float most = 0.5f - inv * (eps + 0x1p-20f * (fmaxf(fabsf(mn[e]), fabsf(mx[e])) + fabsf(m) + 16.f * s));
            constexpr float MAGIC = 12582912.f;
            uint32_t w = 0;
            float far = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = fminf(fmaxf(fmaf(z_of(i, e), inv, off), 0.f), (float)INT4_LEVELS), n = y + MAGIC;
                far = fmaxf(far, fabsf(y - (n - MAGIC)));
                w |= (__float_as_uint(n) & 15u) << (4 * i);
            }
            uint32_t any = __ballot_sync(0xffffffffu, live && !wild && s > 0.f && !(far < most));
            if (any) {
                uint32_t again = 0;
                if (any >> lane & 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float y = fminf(fmaxf(fmaf(z_of(i, e), inv, off), 0.f), (float)INT4_LEVELS);
                        again |= (uint32_t)!(fabsf(y - (y + MAGIC - MAGIC)) < most) << i;
                    }
                }
                while ((any = __ballot_sync(0xffffffffu, again != 0)) != 0) {
                    const int l = __ffs(any) - 1, i = __ffs(__shfl_sync(0xffffffffu, again, l)) - 1;
                    const Dd y = exact((l >> 2) + 8 * e, 32 * g + 8 * (l & 3) + i, std::integral_constant<int, 5>());
                    if (lane == l) {
                        // the nearest threshold decides
                        const float q = fmaf(y.hi - m, inv, -0.5f);
                        const int c = q <= -0.5f ? 0 : q >= INT4_LEVELS - 0.5f ? INT4_LEVELS : int4_code(y, s, m, (int)rintf(q));
                        w = (w & ~(15u << (4 * i))) | (uint32_t)c << (4 * i);
                        again &= again - 1;
                    }
                }
            }
            // ---- rows outside fp32's comfortable range: all in fp64
            uint32_t rows = __ballot_sync(0xffffffffu, wild);
            while (rows) {
                const int base = (__ffs(rows) - 1) & ~3, rw = (base >> 2) + 8 * e;
                double y = 0.0;  // lane = channel of the group
                for (int i = 0; i < D; ++i)
                    y = fma((double)__bfloat162float(sm.A[buf][rw][i]) - (double)sm.mu[i], (double)sm.RT[32 * g + lane][i], y);
                double lo = y, hi = y;
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                    hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                }
                if (__any_sync(0xffffffffu, !isfinite(y))) lo = hi = CUDART_NAN;
                __half a, b;
                int4_params(lo, hi, (double)clip, a, b);
                uint32_t c = (uint32_t)int4_code(y, a, b) << (4 * (lane & 7));
                c |= __shfl_xor_sync(0xffffffffu, c, 1);
                c |= __shfl_xor_sync(0xffffffffu, c, 2);
                c |= __shfl_xor_sync(0xffffffffu, c, 4);
                c = __shfl_sync(0xffffffffu, c, 8 * t);  // the word of channels 8 t ..
                if ((lane & ~3) == base) {
                    w = c;
                    sh[e] = a;
                    mh[e] = b;
                }
                rows &= ~(0xfu << base);
            }
            sm.word[row][t][g] = w;
            if (t == 0) {
                sm.sc[row][g] = sh[e];
                sm.mn[row][g] = mh[e];
            }
        }
        __syncthreads();  // the tile's codes are there
        if (!side) {
            // a token's record: four pieces of codes and one of meta, 16 bytes each
            if (tid < 5 * PF_M) {
                const int row = tid / 5, piece = tid % 5, slot = sm.slot[buf][row];
                if (slot >= 0) {
                    uint8_t* tile = cache + ((size_t)(slot / PAGE) * H_kv + h) * INT4_TILE;
                    const int s = slot % PAGE;
                    if (piece < 4) {
                        *reinterpret_cast<uint4*>(tile + O4_KC + 64 * s + 16 * piece) = *reinterpret_cast<const uint4*>(sm.word[row][piece]);
                    } else {
                        const uint2 a = *reinterpret_cast<const uint2*>(sm.sc[row]), b = *reinterpret_cast<const uint2*>(sm.mn[row]);
                        *reinterpret_cast<uint4*>(tile + O4_KM + 16 * s) = make_uint4(a.x, a.y, b.x, b.y);
                    }
                }
            }
        } else {
            // token pair (2 j, 2 j + 1) of the tile in the two slots of one pair: whole words
            // (thread = eighth of a pair row: channels 32 g + 4 q ..); else halves
            const int j = tid >> 4, q = tid & 15;
            const int sa = sm.slot[buf][2 * j], sb = sm.slot[buf][2 * j + 1];
            const bool pair = sa >= 0 && !(sa & 1) && sb == sa + 1;
            if (pair) {
                uint8_t* tile = cache + ((size_t)(sa / PAGE) * H_kv + h) * INT4_TILE;
                const int s = (sa % PAGE) >> 1;
                if (q < 8) {
                    uint32_t out[4];
                    const uint32_t sel = q & 1 ? 0x7632 : 0x5410;
#pragma unroll
                    for (int gg = 0; gg < 4; ++gg) out[gg] = prmt(sm.word[2 * j][q >> 1][gg], sm.word[2 * j + 1][q >> 1][gg], sel);
                    *reinterpret_cast<uint4*>(tile + O4_VC + 128 * s + 16 * q) = make_uint4(out[0], out[1], out[2], out[3]);
                } else if (q < 10) {
                    const __half(*src2)[NGROUP] = q == 8 ? sm.sc : sm.mn;
                    const uint2 a = *reinterpret_cast<const uint2*>(src2[2 * j]), b = *reinterpret_cast<const uint2*>(src2[2 * j + 1]);
                    *reinterpret_cast<uint4*>(tile + (q == 8 ? O4_VS : O4_VM) + 16 * s) =
                        make_uint4(prmt(a.x, b.x, 0x5410), prmt(a.x, b.x, 0x7632), prmt(a.y, b.y, 0x5410), prmt(a.y, b.y, 0x7632));
                }
            } else {
                for (int e = 0; e < 2; ++e) {
                    const int slot = e ? sb : sa, row = 2 * j + e;
                    if (slot < 0) continue;
                    uint8_t* tile = cache + ((size_t)(slot / PAGE) * H_kv + h) * INT4_TILE;
                    store_word(tile, 1, slot % PAGE, q & 3, q >> 2, sm.word[row][q >> 2][q & 3]);
                    if (q < NGROUP) store_meta(tile, 1, slot % PAGE, q, sm.sc[row][q], sm.mn[row][q]);
                }
            }
        }
    }
}

// ------------------------------------------------------------ read-back
//
// Sixteen threads per (token, KV head, side), a word of eight channels each: one
// fp32 fma and one rounding to bf16 per channel, a 16-byte store.  A thread takes
// four tokens, whose loads are in flight together.

constexpr int DQ_TOK = 4;

__global__ void __launch_bounds__(256)
dequant_int4_kernel(const uint8_t* __restrict__ cache, int64_t num_pages, int H_kv, int n,
                    const int32_t* __restrict__ slot_mapping, __nv_bfloat16* __restrict__ k_rot,
                    __nv_bfloat16* __restrict__ v_rot) {
    griddep_wait();
    griddep_launch_dependents();
    const int side = blockIdx.z, h = blockIdx.y, g = (threadIdx.x >> 2) & 3, t = threadIdx.x & 3;
    __nv_bfloat16* dst = side ? v_rot : k_rot;
    if (!dst) return;
    const int64_t first = (int64_t)blockIdx.x * 16 * DQ_TOK + (threadIdx.x >> 4);
    uint32_t w[DQ_TOK];
    __half sc[DQ_TOK], mn[DQ_TOK];
    int slot[DQ_TOK];
#pragma unroll
    for (int e = 0; e < DQ_TOK; ++e) slot[e] = first + 16 * e < n ? __ldg(slot_mapping + first + 16 * e) : -1;
#pragma unroll
    for (int e = 0; e < DQ_TOK; ++e) {
        w[e] = 0u;
        sc[e] = mn[e] = __ushort_as_half(0);
        if (slot[e] >= 0 && (int64_t)slot[e] < num_pages * PAGE) {
            const int s = slot[e] % PAGE;
            const uint8_t* tile = cache + ((size_t)(slot[e] / PAGE) * H_kv + h) * INT4_TILE;
            if (side) {
                const uint8_t* p = tile + O4_VC + 128 * (s >> 1) + 32 * t + 4 * g + 2 * (s & 1);
                w[e] = (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p)) | (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p + 16)) << 16;
                sc[e] = *reinterpret_cast<const __half*>(tile + O4_VS + int4_vmeta_off(s, g));
                mn[e] = *reinterpret_cast<const __half*>(tile + O4_VM + int4_vmeta_off(s, g));
            } else {
                w[e] = __ldg(reinterpret_cast<const uint32_t*>(tile + O4_KC + 64 * s + 16 * t + 4 * g));
                sc[e] = *reinterpret_cast<const __half*>(tile + O4_KM + 16 * s + 2 * g);
                mn[e] = *reinterpret_cast<const __half*>(tile + O4_KM + 16 * s + 8 + 2 * g);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < DQ_TOK; ++e) {
        if (first + 16 * e >= n) break;
        const float s = __half2float(sc[e]), m = __half2float(mn[e]);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = pack_bf16(__fmaf_rn((float)((w[e] >> (8 * i)) & 15), s, m), __fmaf_rn((float)((w[e] >> (8 * i + 4)) & 15), s, m));
        *reinterpret_cast<uint4*>(dst + ((size_t)(first + 16 * e) * H_kv + h) * D + 32 * g + 8 * t) =
            make_uint4(out[0], out[1], out[2], out[3]);
    }
}

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_int4_tile_bytes(int d) { return d == D ? (size_t)INT4_TILE : 0; }

// Appends of at least this many tokens take the tensor-core kernel.
static constexpr int PREFILL_MIN = 32;

static kvq_status prefill_smem_once() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    kvq_status st = kvq_check_cuda(cudaGetDevice(&dev), "kvq_append_int4: cudaGetDevice");
    if (st != KVQ_OK) return st;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && done[dev]) return KVQ_OK;
    st = kvq_check_cuda(cudaFuncSetAttribute((const void*)append_int4_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)sizeof(PrefillSmem)),
                        "kvq_append_int4 smem attribute");
    if (st == KVQ_OK && dev >= 0 && dev < 64) done[dev] = true;
    return st;
}

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
    for (const void* p : {k, v, (const void*)R_k, (const void*)R_v, (const void*)cache})
        if (reinterpret_cast<uintptr_t>(p) % 16)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_append_int4: k, v, R_k, R_v and cache need to be 16-byte aligned");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto kb = static_cast<const __nv_bfloat16*>(k), vb = static_cast<const __nv_bfloat16*>(v);
    uint8_t* const cb = static_cast<uint8_t*>(cache);
    if (n_tok < PREFILL_MIN)
        return kvq_check_cuda(launch_pdl(append_int4_kernel, dim3(n_tok, H_kv, 2), dim3(512), 0, st, kb, vb, n_tok, H_kv,
                                         slot_mapping, mu_k, R_k, R_v, cb, num_pages, err_count, clip),
                              "kvq_append_int4 launch");
    const kvq_status sa = prefill_smem_once();
    if (sa != KVQ_OK) return sa;
    // two CTAs per SM in all, each with a stride of its (head, side)'s tiles
    const int tiles = (n_tok + PF_M - 1) / PF_M, most = (2 * kvq_device_sm_count() + 2 * H_kv - 1) / (2 * H_kv);
    return kvq_check_cuda(launch_pdl(append_int4_prefill_kernel, dim3(tiles < most ? tiles : most, H_kv, 2), dim3(128),
                                     sizeof(PrefillSmem), st, kb, vb, n_tok, H_kv, slot_mapping, mu_k, R_k, R_v, cb, num_pages,
                                     err_count, clip),
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
    for (const void* p : {cache, (const void*)k_rot, (const void*)v_rot})
        if (reinterpret_cast<uintptr_t>(p) % 16)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "kvq_dequant_int4: cache, k_rot and v_rot need to be 16-byte aligned");
    const int blocks = (int)(((int64_t)n + 16 * DQ_TOK - 1) / (16 * DQ_TOK));
    return kvq_check_cuda(launch_pdl(dequant_int4_kernel, dim3(blocks, H_kv, 2), dim3(256), 0, static_cast<cudaStream_t>(stream),
                                     static_cast<const uint8_t*>(cache), num_pages, H_kv, n, slot_mapping,
                                     static_cast<__nv_bfloat16*>(k_rot), static_cast<__nv_bfloat16*>(v_rot)),
                          "kvq_dequant_int4 launch");
}
