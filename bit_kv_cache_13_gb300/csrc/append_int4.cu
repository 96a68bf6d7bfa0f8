// Quantise-on-append and read-back of the rotated INT4 KV cache.
//
// z = (k - mu) R_k, w = v R_v, then 16 levels per group of 32 rotated channels
// with an fp16 scale and min.  Codes, scales and mins are those of the exact
// rotated vectors, whichever kernel writes them: each kernel forms the rotated
// values to within a bound, and where a rounding or a threshold lies within that
// bound of a value (a few groups in a hundred) it forms the value exactly.
#include <algorithm>
#include <cstddef>
#include <mutex>

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

// Token t's slot; -1 to skip it, -2 for one that is skipped and counted.
__device__ __forceinline__ int append_slot(const AppendInt4& a, int64_t t) {
    const int slot = __ldg(a.slot_mapping + t);
    if (slot == -1) return -1;
    bool ok = slot >= 0 && (int64_t)slot < a.num_pages * PAGE;
    if (a.positions) ok = ok && (unsigned)__ldg(a.positions + t) < (unsigned)a.max_pos;
    return ok ? slot : -2;
}

// ------------------------------------------------------------ a few tokens
//
// One CTA of 512 threads per (token, KV head, side): thread (channel, quarter)
// sums 32 products in an unevaluated pair of fp32 values, so the rotated values are
// exact to about 46 bits and no second look is taken.  Bound by its chain of
// latencies: one row of R_k per thread and quarter in flight (one token of eight heads,
// with the read-back in a second kernel, 4.5 us).

__global__ void __launch_bounds__(512)
append_int4_kernel(const __grid_constant__ AppendInt4 a) {
    __shared__ float xs[D], xl[D], n2s[4];
    __shared__ Dd part[4][D];
    const int t = blockIdx.x, h = blockIdx.y, side = blockIdx.z, tid = threadIdx.x;
    const int j = tid & (D - 1), quarter = tid >> 7, lane = tid & 31, g = (tid >> 5) & 3;
    const float* R = (side ? a.R_v : a.R_k) + (size_t)h * D * D + (size_t)32 * quarter * D + j;
    prefetch_l2(R - j + (size_t)(j >> 2) * D + 32 * (j & 3));  // the quarter's 32 rows, four lines each
    griddep_wait();
    griddep_launch_dependents();
    const int slot = append_slot(a, t);
    float rr[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) rr[i] = __ldg(R + (size_t)i * D);
    if (slot < 0) {
        if (slot != -1 && tid == 0 && h == 0 && side == 0 && a.err_count) atomicAdd(a.err_count, 1);
        return;
    }
    if (quarter == 0) {
        const size_t row = (size_t)t * (side ? a.v_stride : a.k_stride) + h * D + j;
        const float x = __bfloat162float((side ? a.v : a.k)[row]);
        const float m = side ? 0.f : __ldg(a.mu_k + (size_t)h * D + j);
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
    Dd z = part[0][j], y = part[2][j];
    dd_add(z, part[1][j]);
    dd_add(y, part[3][j]);
    dd_add(z, y);
    z = dd_norm(z);
    // (a matrix's large entries can take the pairs out of range, or hold what is not finite)
    if (!wild && __all_sync(0xffffffffu, isfinite(z.hi))) {
        Dd mn = z, mx = z;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const Dd a = {__shfl_xor_sync(0xffffffffu, mn.hi, o), __shfl_xor_sync(0xffffffffu, mn.lo, o)};
            const Dd b = {__shfl_xor_sync(0xffffffffu, mx.hi, o), __shfl_xor_sync(0xffffffffu, mx.lo, o)};
            if (dd_less(a, mn)) mn = a;
            if (dd_less(mx, b)) mx = b;
        }
        int4_params(mn, mx, a.clip, sh, mh);
        const float s = __half2float(sh), m = __half2float(mh);
        // the nearest threshold decides between two codes (past the ends, and for s = 0, the end)
        const float q = s > 0.f ? fmaf(z.hi - m, 1.f / s, -0.5f) : -1.f;
        code = q <= -0.5f ? 0 : q >= INT4_LEVELS - 0.5f ? INT4_LEVELS : int4_code(z, s, m, (int)rintf(q));
    } else {  // all in fp64
        const float* Rw = (side ? a.R_v : a.R_k) + (size_t)h * D * D + j;
        double w = 0.0;
        for (int i = 0; i < D; ++i) w = fma((double)xs[i] + (double)xl[i], (double)__ldg(Rw + (size_t)i * D), w);
        double lo = w, hi = w;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (__any_sync(0xffffffffu, !isfinite(w))) lo = hi = CUDART_NAN;
        int4_params(lo, hi, (double)a.clip, sh, mh);
        code = int4_code(w, sh, mh);
    }
    // the eight codes of a word sit in eight neighbouring lanes
    uint32_t w = (uint32_t)code << (4 * (lane & 7));
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    uint8_t* tile = a.cache + ((size_t)(slot / PAGE) * a.H_kv + h) * INT4_TILE;
    if ((lane & 7) == 0) store_word(tile, side, slot % PAGE, g, lane >> 3, w);
    if (lane == 0) store_meta(tile, side, slot % PAGE, g, sh, mh);
}

// ------------------------------------------------------------ prefill
//
// The rotation on the tensor cores.  The inputs are bf16 and so exact operands; R
// enters as three bf16 parts (8 bits each: its fp32 value, exactly), smallest first,
// into one fp32 accumulator, and the centre is subtracted after the rotation (z = k R
// - mu R, mu R formed once per CTA).  The parts stand in shared memory in operand
// order; one CTA per SM holds those of one (KV head, side), and its four workers of
// four warps go their own ways through tiles of 32 tokens: warp g of a worker forms
// group g's 32 channels of them.  With the columns of the product in the order
// channel 8 t + 2 i + e = column 2 t + e of its eight columns' set i, the accumulators
// of a lane are the eight codes of one word of the key record.
//
// A matrix instruction's sum, as its results show (an integer model gives all of 6 M of
// them to the bit): every term, the accumulator too, is cut off at 2^-25 of 2^E, E the
// largest exponent among the terms (of a product, the sum of its factors'), and their sum
// at 24 bits, both toward zero.  With an accumulator that has grown, each of a step's 16
// products would lose 2^-25 of it; so every step of R's largest part starts from zero, and
// the steps are added in fp32.  With S = |R_j| |k| >= sum_i |R_ij k_i| and K_b the largest
// |k_i| of step b's 16 channels, in units of 2^-23:
//   16 terms a step cut at 2^-25 max |R| K_b          4 max |R| sum_b K_b
//   the steps' sums cut at 24 bits                    S
//   adding steps in pairs, and the pairs              (1/2 + 4/2) S
//   the smaller parts (2^-8 S), 16 steps of 17 terms  8 (17/4 + 1) 2^-8 S < 0.2 S
//   rounding mu R, subtracting it                     1/2 S + |R_j| |mu|
//   rounding ends +- twice the bound                  1/4 S
// which is at most PF_NORM |R_j| (|k| + |mu|) + PF_MOST max |R| sum_b K_b with R_j the
// largest column.  (One chain of the 8 steps would be 42 S.)
// Groups or codes that the bound leaves open (a few groups in a hundred, one
// code in ten thousand) take exact dot products in pairs of fp32 values, a worker's
// together in one list: fp64 is 64 times slower than fp32 here, and a first form of
// these second looks in fp64 took most of the kernel's time.
//
// 32K tokens of eight heads: 263 us, bound by the instructions of the epilogue and the
// second looks (50 % issue, four warps per scheduler at 128 registers, the tensor pipe
// 30 %).
constexpr int PF_WORKERS = 4, PF_M = 32;  // tokens of a worker's tile
constexpr float PF_NORM = 4.625f * 0x1p-23f, PF_MOST = 4.125f * 0x1p-23f;
constexpr int PF_KEY_COST = 6, PF_VALUE_COST = 5;  // of a tile's time (more keys are looked at twice: the centre is in their bound)
constexpr int PF_A = D + 8;               // padded rows, in elements

struct __align__(16) PrefillWorker {
    __align__(16) __nv_bfloat16 A[2][PF_M][PF_A];
    __align__(16) uint32_t word[PF_M][4][4];  // the tile's codes [token][t][g]
    __align__(16) __half sc[PF_M][NGROUP];
    __align__(16) __half mn[PF_M][NGROUP];
    uint32_t open_cand[PF_M * NGROUP];        // groups whose parameters are open: channels to look at, and
    uint16_t open_id[PF_M * NGROUP];          // row << 4 | group << 2 | what is open
    float eps[PF_M];                          // the bound on the rows' errors; -1: a row for fp64
    int slot[2][PF_M];
    int n_open;
};
struct __align__(16) PrefillSmem {
    __align__(16) uint2 R[3][NGROUP][4][8][32];  // parts as operands: [part][group][set][K step][lane]
    __align__(16) float mu[D];                // the centre (0 for values)
    __align__(16) float c[D];                 // mu R (0 for values)
    __align__(16) Dd c_exact[D];
    float m2[4], col2[PF_WORKERS * 4], col_most[PF_WORKERS * 4], mu_norm;
    float bound, bound_most;                  // PF_NORM times the largest column's norm (-1: fp64), PF_MOST times the largest entry
    PrefillWorker w[PF_WORKERS];
};
static_assert(offsetof(PrefillSmem, R) % 16 == 0 && offsetof(PrefillSmem, mu) % 16 == 0 && offsetof(PrefillSmem, c) % 16 == 0 &&
                  offsetof(PrefillSmem, w) % 16 == 0 && sizeof(PrefillWorker) % 16 == 0 && offsetof(PrefillWorker, A) % 16 == 0 &&
                  offsetof(PrefillWorker, word) % 16 == 0 && offsetof(PrefillWorker, sc) % 8 == 0 &&
                  offsetof(PrefillWorker, mn) % 8 == 0 && (PF_A * 2) % 16 == 0,
              "wide accesses to shared memory are aligned");
static_assert(sizeof(PrefillSmem) <= 227 * 1024, "prefill shared memory above 227 KB");

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The product alone.
__device__ __forceinline__ void mma0_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// x + y, two fp32 sums in one instruction.
__device__ __forceinline__ void add2(float& x0, float& x1, float y0, float y1) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
        : "+f"(x0), "+f"(x1)
        : "f"(y0), "f"(y1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Takes the nearest bf16 value off x.
__device__ __forceinline__ float bf16_part(float& x) {
    const float p = __bfloat162float(__float2bfloat16_rn(x));
    x = x - p;  // exact
    return p;
}

// Inputs 16 ks + 2 q, + 1, + 8, + 9 of channel ch's column of R, from its parts: exact sums.
__device__ __forceinline__ float4 prefill_column(const PrefillSmem& sm, int ch, int ks, int q) {
    const int c = ch & 31, at = 4 * (2 * (c >> 3) + (c & 1)) + q;
    const uint2 a = sm.R[0][ch >> 5][(c >> 1) & 3][ks][at], b = sm.R[1][ch >> 5][(c >> 1) & 3][ks][at],
                d = sm.R[2][ch >> 5][(c >> 1) & 3][ks][at];
    return make_float4((bf16_lo(a.x) + bf16_lo(b.x)) + bf16_lo(d.x), (bf16_hi(a.x) + bf16_hi(b.x)) + bf16_hi(d.x),
                       (bf16_lo(a.y) + bf16_lo(b.y)) + bf16_lo(d.y), (bf16_hi(a.y) + bf16_hi(b.y)) + bf16_hi(d.y));
}

// k . R[:, ch] - (mu R)[ch] (or v . R[:, ch]) of a row A: sixteen lanes, two times four
// inputs each; all of them get the sum.  (Not inlined: the kernel's loop has to stay
// within the instruction cache.  With these sums and the fp64 path unrolled into it, a
// warp waited 4.4 cycles for each instruction's fetch.)
__device__ __noinline__ Dd prefill_exact(const PrefillSmem& sm, const __nv_bfloat16* A, int ch) {
    const int lane = threadIdx.x & 31;
    Dd s[2] = {};
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int e = 16 * y + (lane & 15), i0 = 16 * (e >> 2) + 2 * (e & 3);
        const uint32_t xa = *reinterpret_cast<const uint32_t*>(A + i0), xb = *reinterpret_cast<const uint32_t*>(A + i0 + 8);
        const float4 rv = prefill_column(sm, ch, e >> 2, e & 3);
        dd_fma(s[0], bf16_lo(xa), 0.f, rv.x);
        dd_fma(s[1], bf16_hi(xa), 0.f, rv.y);
        dd_fma(s[0], bf16_lo(xb), 0.f, rv.z);
        dd_fma(s[1], bf16_hi(xb), 0.f, rv.w);
    }
    dd_add(s[0], s[1]);
#pragma unroll
    for (int o = 8; o; o >>= 1) {
        const Dd y = {__shfl_xor_sync(0xffffffffu, s[0].hi, o), __shfl_xor_sync(0xffffffffu, s[0].lo, o)};
        dd_add(s[0], y);
    }
    // (the butterfly adds in another order in each lane: take the group's first)
    s[0].hi = __shfl_sync(0xffffffffu, s[0].hi, lane & 16);
    s[0].lo = __shfl_sync(0xffffffffu, s[0].lo, lane & 16);
    const Dd c = sm.c_exact[ch];
    dd_add(s[0], Dd{-c.hi, -c.lo});
    return dd_norm(s[0]);
}

// A row all in fp64, lane = channel of group g: its code, scale and min.  (From R itself:
// a bf16 part of its largest numbers would be infinite.)
__device__ __noinline__ int prefill_wild(const PrefillSmem& sm, const float* R, const __nv_bfloat16* A, int g, float clip, __half& sh, __half& mh) {
    double y = 0.0;
#pragma unroll 4
    for (int i = 0; i < D; ++i)
        y = fma((double)__bfloat162float(A[i]) - (double)sm.mu[i], (double)__ldg(R + (size_t)i * D + 32 * g + (threadIdx.x & 31)), y);
    double lo = y, hi = y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (__any_sync(0xffffffffu, !isfinite(y))) lo = hi = CUDART_NAN;
    int4_params(lo, hi, (double)clip, sh, mh);
    return int4_code(y, sh, mh);
}

__global__ void __launch_bounds__(PF_WORKERS * 128, 1)
append_int4_prefill_kernel(const __grid_constant__ AppendInt4 args, int key_ctas) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    PrefillSmem& sm = *reinterpret_cast<PrefillSmem*>(smem_raw);
    const int h = blockIdx.y, side = blockIdx.x >= key_ctas, worker = threadIdx.x >> 7, tid = threadIdx.x & 127;
    const int g = tid >> 5, lane = tid & 31, r = lane >> 2, t = lane & 3;
    PrefillWorker& wk = sm.w[worker];
    const float* R = (side ? args.R_v : args.R_k) + (size_t)h * D * D;
    prefetch_l2(R + 32 * threadIdx.x);  // (512 lines)
    griddep_wait();
    griddep_launch_dependents();

    const int n_tok = args.n_tok, tiles = (n_tok + PF_M - 1) / PF_M, ctas = side ? gridDim.x - key_ctas : key_ctas, stride = ctas * PF_WORKERS;
    const __nv_bfloat16* src = (side ? args.v : args.k) + h * D;
    const int64_t src_stride = side ? args.v_stride : args.k_stride;
    const float clip = args.clip;
    uint8_t* const cache = args.cache;
    const int H_kv = args.H_kv;
    auto worker_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(worker + 1) : "memory"); };
    auto fetch = [&](int x, int buf) {  // tile x: 512 pieces of 16 bytes, and its slots
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = tid + 128 * e, row = p >> 4, col = 8 * (p & 15);
            const int64_t tok = min((int64_t)x * PF_M + row, (int64_t)n_tok - 1);  // (rows past the end repeat the last)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&wk.A[buf][row][col])),
                         "l"(src + tok * src_stride + col)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (tid < PF_M) {
            const int64_t tok = (int64_t)x * PF_M + tid;
            int s = tok < n_tok ? append_slot(args, tok) : -1;
            if (s < -1) {
                if (h == 0 && side == 0 && args.err_count) atomicAdd(args.err_count, 1);
                s = -1;
            }
            wk.slot[buf][tid] = s;
        }
    };
    const int x_first = blockIdx.x - (side ? key_ctas : 0) + worker * ctas;  // (few tiles: on as many SMs as there are)
    if (x_first < tiles) fetch(x_first, 0);
    // R's parts as operands: column n of set i of a group is channel 8 (n / 2) + 2 i + n % 2 of it
#pragma unroll 2
    for (int y = threadIdx.x; y < NGROUP * 4 * 8 * 32; y += PF_WORKERS * 128) {
        const int ks = (y >> 5) & 7, i = (y >> 8) & 3, gg = y >> 10;  // (r, t: this lane's column and rows)
        const float* p = R + (size_t)(16 * ks + 2 * t) * D + 32 * gg + 8 * (r >> 1) + 2 * i + (r & 1);
        float a = __ldg(p), b = __ldg(p + D), c = __ldg(p + 8 * D), d = __ldg(p + 9 * D);
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const float a0 = bf16_part(a), b0 = bf16_part(b), c0 = bf16_part(c), d0 = bf16_part(d);
            sm.R[q][gg][i][ks][lane] = make_uint2(pack_bf16(a0, b0), pack_bf16(c0, d0));
        }
    }
    if (threadIdx.x < D) {
        const float m = side ? 0.f : __ldg(args.mu_k + (size_t)h * D + threadIdx.x);
        sm.mu[threadIdx.x] = m;
        float m2 = m * m;
#pragma unroll
        for (int o = 16; o; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
        if (lane == 0) sm.m2[g] = m2;
    }
    __syncthreads();
    {   // the columns' norms and mu R: four neighbouring threads a channel
        const int ch = threadIdx.x >> 2, q = threadIdx.x & 3;
        Dd s[2] = {};
        float n2 = 0.f, most = 0.f;
#pragma unroll 2
        for (int ks = 0; ks < 8; ++ks) {
            const float4 x = prefill_column(sm, ch, ks, q);
            n2 = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, fmaf(x.w, x.w, n2))));
            most = fmaxf(fmaxf(most, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
            if (side) continue;
            dd_fma(s[0], sm.mu[16 * ks + 2 * q], 0.f, x.x);
            dd_fma(s[1], sm.mu[16 * ks + 2 * q + 1], 0.f, x.y);
            dd_fma(s[0], sm.mu[16 * ks + 2 * q + 8], 0.f, x.z);
            dd_fma(s[1], sm.mu[16 * ks + 2 * q + 9], 0.f, x.w);
        }
        dd_add(s[0], s[1]);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            const Dd y = {__shfl_xor_sync(0xffffffffu, s[0].hi, o), __shfl_xor_sync(0xffffffffu, s[0].lo, o)};
            dd_add(s[0], y);
        }
        if (q == 0) {
            sm.c[ch] = s[0].hi + s[0].lo;
            sm.c_exact[ch] = dd_norm(s[0]);
        }
        n2 += __shfl_xor_sync(0xffffffffu, n2, 1);
        n2 += __shfl_xor_sync(0xffffffffu, n2, 2);
        const int wild = __syncthreads_or(!(n2 < 0x1p100f));  // large numbers, or NaN: all rows in fp64
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            n2 = fmaxf(n2, __shfl_xor_sync(0xffffffffu, n2, o));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        }
        if (lane == 0) {
            sm.col2[threadIdx.x >> 5] = n2;
            sm.col_most[threadIdx.x >> 5] = most;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 0; w < PF_WORKERS * 4; ++w) {
                n2 = fmaxf(n2, sm.col2[w]);
                most = fmaxf(most, sm.col_most[w]);
            }
            sm.bound = wild ? -1.f : PF_NORM * sqrtf(n2);
            sm.bound_most = PF_MOST * most;
            sm.mu_norm = sqrtf((sm.m2[0] + sm.m2[1]) + (sm.m2[2] + sm.m2[3]));
        }
    }
    __syncthreads();  // the last barrier of the whole CTA

    int buf = 0;
#pragma unroll 1
    for (int x = x_first; x < tiles; x += stride, buf ^= 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        worker_sync();  // the tile is there; the last one's words are written out
        {   // the rows' bounds: 4 threads a row, two steps' channels each
            const int row = tid >> 2, q = tid & 3;
            const uint4* p = reinterpret_cast<const uint4*>(&wk.A[buf][row][32 * q]);
            float n2 = 0.f, most = 0.f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 v = p[2 * (b ^ (q >> 1)) + e];  // (no two of eight lanes in the same banks)
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        n2 = fmaf(bf16_lo(w[y]), bf16_lo(w[y]), fmaf(bf16_hi(w[y]), bf16_hi(w[y]), n2));
                        top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[y])));
                    }
                }
                most += fmaxf(__low2float(top), __high2float(top));
            }
            n2 += __shfl_xor_sync(0xffffffffu, n2, 1);
            n2 += __shfl_xor_sync(0xffffffffu, n2, 2);
            most += __shfl_xor_sync(0xffffffffu, most, 1);
            most += __shfl_xor_sync(0xffffffffu, most, 2);
            if (q == 0)
                wk.eps[row] = sm.bound < 0.f || int4_wild(n2 + sm.mu_norm * sm.mu_norm) ? -1.f : fmaf(sm.bound, sqrtf(n2) + sm.mu_norm, sm.bound_most * most);
            if (tid == 0) wk.n_open = 0;
        }
        if (x + stride < tiles) fetch(x + stride, buf ^ 1);

        float acc[2][4][4];  // [16 tokens][set][..]
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.f;
        const uint32_t a_addr = smem_u32(&wk.A[buf][lane & 15][8 * (lane >> 4)]);
        auto load_a = [&](int ks, uint32_t (&a)[2][4]) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                             : "=r"(a[m][0]), "=r"(a[m][1]), "=r"(a[m][2]), "=r"(a[m][3])
                             : "r"(a_addr + 32 * ks + 16 * PF_A * 2 * m));
        };
#pragma unroll 1
        for (int p = 2; p >= 1; --p)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t a[2][4];
                load_a(ks, a);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 f = sm.R[p][g][i][ks][lane];
                    mma_bf16(acc[0][i], a[0], f.x, f.y);
                    mma_bf16(acc[1][i], a[1], f.x, f.y);
                }
            }
#pragma unroll
        for (int ks = 0; ks < 8; ks += 2) {
            uint32_t a[2][4], b[2][4];
            load_a(ks, a);
            load_a(ks + 1, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint2 f = sm.R[0][g][i][ks][lane], h2 = sm.R[0][g][i][ks + 1][lane];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float d0[4], d1[4];
                    mma0_bf16(d0, a[m], f.x, f.y);
                    mma0_bf16(d1, b[m], h2.x, h2.y);
                    add2(d0[0], d0[1], d1[0], d1[1]);
                    add2(d0[2], d0[3], d1[2], d1[3]);
                    add2(acc[m][i][0], acc[m][i][1], d0[0], d0[1]);
                    add2(acc[m][i][2], acc[m][i][3], d0[2], d0[3]);
                }
            }
        }
        worker_sync();  // the bounds are there

        // row set q = 2 m + e: rows 16 m + 8 e + r; its channel 32 g + 8 t + i of this lane
        auto row_of = [&](int q) { return 16 * (q >> 1) + 8 * (q & 1) + r; };
        auto z_of = [&](int i, int q) -> float& { return acc[q >> 1][i >> 1][2 * (q & 1) + (i & 1)]; };
        if (side == 0) {
            const float4 ca = *reinterpret_cast<const float4*>(&sm.c[32 * g + 8 * t]), cb = *reinterpret_cast<const float4*>(&sm.c[32 * g + 8 * t + 4]);
            const float cc[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 8; ++i) z_of(i, q) -= cc[i];
        }
        // ---- each row's parameters; open ones go on the worker's list
        float top[4];  // largest magnitude of the group
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float mn = z_of(0, q), mx = mn;
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                mn = fminf(mn, z_of(i, q));
                mx = fmaxf(mx, z_of(i, q));
            }
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, 2));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            top[q] = fmaxf(fabsf(mn), fabsf(mx));
            const float eps = wk.eps[row_of(q)];
            __half sh, mh;
            const int near = int4_params_near(mn, mx, clip, eps, sh, mh);
            const bool open = near && eps >= 0.f && wk.slot[buf][row_of(q)] >= 0;
            if (t == 0) {
                wk.sc[row_of(q)][g] = sh;
                wk.mn[row_of(q)][g] = mh;
            }
            if (__any_sync(0xffffffffu, open)) {
                // every value that could be the smallest (the largest, where the scale is open)
                const float low = mn + 2.f * eps, high = near > 1 ? mx - 2.f * eps : CUDART_INF_F;
                uint32_t c = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) c |= (uint32_t)(z_of(i, q) <= low || z_of(i, q) >= high) << i;
                c <<= 8 * t;
                c |= __shfl_xor_sync(0xffffffffu, c, 1);
                c |= __shfl_xor_sync(0xffffffffu, c, 2);
                if (open && t == 0) {
                    const int at = atomicAdd(&wk.n_open, 1);
                    wk.open_cand[at] = c;
                    wk.open_id[at] = (uint16_t)(row_of(q) << 4 | g << 2 | near);
                }
            }
        }
        worker_sync();  // the list is complete
        const int n_open = wk.n_open;
        if (n_open > 0) {
            // a warp takes a group at a time, two values at a time
#pragma unroll 1
            for (int y = g; y < n_open; y += 4) {
                uint32_t c = wk.open_cand[y];
                const int id = wk.open_id[y], row = id >> 4, gg = id >> 2 & 3;
                Dd lo = {CUDART_INF_F, 0.f}, hi = {-CUDART_INF_F, 0.f};
#pragma unroll 1
                while (c) {
                    const int first = __ffs(c) - 1;
                    c &= c - 1;
                    const int second = c ? __ffs(c) - 1 : first;
                    c &= c - 1;
                    const Dd z = prefill_exact(sm, wk.A[buf][row], 32 * gg + (lane < 16 ? first : second));
                    if (dd_less(z, lo)) lo = z;
                    if (dd_less(hi, z)) hi = z;
                }
                const Dd l2 = {__shfl_xor_sync(0xffffffffu, lo.hi, 16), __shfl_xor_sync(0xffffffffu, lo.lo, 16)};
                const Dd h2 = {__shfl_xor_sync(0xffffffffu, hi.hi, 16), __shfl_xor_sync(0xffffffffu, hi.lo, 16)};
                if (dd_less(l2, lo)) lo = l2;
                if (dd_less(hi, h2)) hi = h2;
                __half sh, mh;
                int4_params(lo, hi, clip, sh, mh);
                if (lane == 0) {
                    if (id & 2) wk.sc[row][gg] = sh;
                    wk.mn[row][gg] = mh;
                }
            }
            worker_sync();
        } else {
            __syncwarp();  // (a warp's parameters are its own)
        }
        uint32_t agains = 0, wilds = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = row_of(q);
            const float eps = wk.eps[row];
            // ---- codes: 15 times z's place in [min, min + 15 scale], rounded by adding 1.5 2^23; what
            // that leaves says how near a threshold is (2^-21 of the terms and 2^-19: twice what the
            // roundings of the place and its product make)
            const float s = __half2float(wk.sc[row][g]), m = __half2float(wk.mn[row][g]), inv = s > 0.f ? 1.f / s : 0.f;
            const float inv15 = inv * (1.f / INT4_LEVELS), off15 = -m * inv15;
            const float most = 0.5f - 0x1p-19f - inv * (eps + 0x1p-21f * (top[q] + fabsf(m)));
            constexpr float MAGIC = 12582912.f;
            uint32_t w = 0;
            float far = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = __saturatef(fmaf(z_of(i, q), inv15, off15)), n = fmaf(y, (float)INT4_LEVELS, MAGIC);
                far = fmaxf(far, fabsf(fmaf(y, (float)INT4_LEVELS, MAGIC - n)));
                w += __float_as_uint(n) << (4 * i);  // (MAGIC's bits come off below)
            }
            w -= 0x4b400000u * 0x11111111u;  // (1.5 2^23 as bits, times 16^0 + .. + 16^7)
            wk.word[row][t][g] = w;
            const bool live = wk.slot[buf][row] >= 0;
            wilds |= (uint32_t)(live && eps < 0.f) << q;
            if (live && eps >= 0.f && s > 0.f && !(far < most)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = __saturatef(fmaf(z_of(i, q), inv15, off15)), n = fmaf(y, (float)INT4_LEVELS, MAGIC);
                    agains |= (uint32_t)!(fabsf(fmaf(y, (float)INT4_LEVELS, MAGIC - n)) < most) << (8 * q + i);
                }
            }
        }
        // ---- codes that a threshold is near to: the exact value and the nearest threshold
        uint32_t any;
#pragma unroll 1
        while ((any = __ballot_sync(0xffffffffu, agains != 0)) != 0) {
            const int l = __ffs(any) - 1, bit = __ffs(__shfl_sync(0xffffffffu, agains, l)) - 1, q = bit >> 3, i = bit & 7;
            const int row = row_of(q) - r + (l >> 2);
            const Dd y = prefill_exact(sm, wk.A[buf][row], 32 * g + 8 * (l & 3) + i);
            if (lane == l) {
                const float s = __half2float(wk.sc[row][g]), m = __half2float(wk.mn[row][g]), z = fmaf(y.hi - m, 1.f / s, -0.5f);
                const int c = z <= -0.5f ? 0 : z >= INT4_LEVELS - 0.5f ? INT4_LEVELS : int4_code(y, s, m, (int)rintf(z));
                wk.word[row][t][g] = (wk.word[row][t][g] & ~(15u << (4 * i))) | (uint32_t)c << (4 * i);
                agains &= agains - 1;
            }
        }
        // ---- rows outside fp32's comfortable range: all in fp64
#pragma unroll 1
        while ((any = __ballot_sync(0xffffffffu, wilds != 0)) != 0) {
            const int l = __ffs(any) - 1, q = __ffs(__shfl_sync(0xffffffffu, wilds, l)) - 1, row = row_of(q) - r + (l >> 2);
            __half sh, mh;
            uint32_t c = (uint32_t)prefill_wild(sm, R, wk.A[buf][row], g, clip, sh, mh) << (4 * (lane & 7));
            c |= __shfl_xor_sync(0xffffffffu, c, 1);
            c |= __shfl_xor_sync(0xffffffffu, c, 2);
            c |= __shfl_xor_sync(0xffffffffu, c, 4);
            c = __shfl_sync(0xffffffffu, c, 8 * t);  // the word of channels 8 t ..
            if ((lane >> 2) == (l >> 2)) {
                wk.word[row][t][g] = c;
                if (t == 0) {
                    wk.sc[row][g] = sh;
                    wk.mn[row][g] = mh;
                }
                wilds &= ~(1u << q);
            }
        }
        worker_sync();  // the tile's codes are there
        if (!side) {
            // a token's record: four pieces of codes and one of meta, 16 bytes each
            for (int y = tid; y < 5 * PF_M; y += 128) {
                const int row = y / 5, piece = y % 5, slot = wk.slot[buf][row];
                if (slot < 0) continue;
                uint8_t* tile = cache + ((size_t)(slot / PAGE) * H_kv + h) * INT4_TILE;
                const int s = slot % PAGE;
                if (piece < 4) {
                    *reinterpret_cast<uint4*>(tile + O4_KC + 64 * s + 16 * piece) = *reinterpret_cast<const uint4*>(wk.word[row][piece]);
                } else {
                    const uint2 a = *reinterpret_cast<const uint2*>(wk.sc[row]), b = *reinterpret_cast<const uint2*>(wk.mn[row]);
                    *reinterpret_cast<uint4*>(tile + O4_KM + 16 * s) = make_uint4(a.x, a.y, b.x, b.y);
                }
            }
        } else {
            // token pair (2 j, 2 j + 1) of the tile in the two slots of one pair: whole words
            // (thread = eighth of a pair row: channels 32 g + 4 q ..); else halves
#pragma unroll
            for (int rep = 0; rep < 2; ++rep) {
                const int j = 8 * rep + (tid >> 4), q = tid & 15;
                const int sa = wk.slot[buf][2 * j], sb = wk.slot[buf][2 * j + 1];
                if (sa >= 0 && !(sa & 1) && sb == sa + 1) {
                    uint8_t* tile = cache + ((size_t)(sa / PAGE) * H_kv + h) * INT4_TILE;
                    const int s = (sa % PAGE) >> 1;
                    if (q < 8) {
                        uint32_t out[4];
                        const uint32_t sel = q & 1 ? 0x7632 : 0x5410;
#pragma unroll
                        for (int gg = 0; gg < 4; ++gg) out[gg] = prmt(wk.word[2 * j][q >> 1][gg], wk.word[2 * j + 1][q >> 1][gg], sel);
                        *reinterpret_cast<uint4*>(tile + O4_VC + 128 * s + 16 * q) = make_uint4(out[0], out[1], out[2], out[3]);
                    } else if (q < 10) {
                        const __half(*from)[NGROUP] = q == 8 ? wk.sc : wk.mn;
                        const uint2 a = *reinterpret_cast<const uint2*>(from[2 * j]), b = *reinterpret_cast<const uint2*>(from[2 * j + 1]);
                        *reinterpret_cast<uint4*>(tile + (q == 8 ? O4_VS : O4_VM) + 16 * s) =
                            make_uint4(prmt(a.x, b.x, 0x5410), prmt(a.x, b.x, 0x7632), prmt(a.y, b.y, 0x5410), prmt(a.y, b.y, 0x7632));
                    }
                } else {
                    for (int e = 0; e < 2; ++e) {
                        const int slot = e ? sb : sa, row = 2 * j + e;
                        if (slot < 0) continue;
                        uint8_t* tile = cache + ((size_t)(slot / PAGE) * H_kv + h) * INT4_TILE;
                        store_word(tile, 1, slot % PAGE, q & 3, q >> 2, wk.word[row][q >> 2][q & 3]);
                        if (q < NGROUP) store_meta(tile, 1, slot % PAGE, q, wk.sc[row][q], wk.mn[row][q]);
                    }
                }
            }
        }
    }
}

// ------------------------------------------------------------ read-back
//
// Sixteen threads per (token, KV head, side), a word of eight channels each: one
// fp32 fma and one rounding to bf16 per channel, a 16-byte store.  A thread takes
// four tokens, whose loads are in flight together.  Bound by its stores: 32K tokens of
// eight heads 34 us, 134 MB written and 42 MB read, 5.1 TB/s.

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

// Token-heads from which on the tensor-core kernel is taken, for each wave of its CTAs:
// it starts in about 12 us a wave (R's operand parts), the few-token kernel takes 0.03 us a
// token-head.  With the read-back: 33 tokens of 8 heads 13.9 against 11.2 us, 64 tokens of
// one head 13.1 against 5.2, 128 of two 14.5 against 11.6, 64 of 8 14.4 against 17.9, 128 of
// 8 15.1 against 30.8.
static constexpr int PREFILL_MIN = 400;

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

kvq_status kvq_append_int4_args(const char* fn, const AppendInt4& a, int d) {
    if (d != D) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: d=%d (only 128)", fn, d);
    if (a.n_tok < 0 || a.H_kv <= 0 || a.num_pages <= 0)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: n_tok=%d H_kv=%d num_pages=%lld", fn, a.n_tok, a.H_kv,
                             (long long)a.num_pages);
    if (a.H_kv > 65535) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: H_kv=%d too large", fn, a.H_kv);
    if (!(a.clip > 0.f && a.clip <= 1.f))
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: clip ratio %g outside (0, 1]", fn, (double)a.clip);
    if (a.n_tok == 0) return KVQ_OK;
    if (!a.k || !a.v || !a.slot_mapping || !a.mu_k || !a.R_k || !a.R_v || !a.cache)
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void* p : {(const void*)a.k, (const void*)a.v, (const void*)a.R_k, (const void*)a.R_v, (const void*)a.cache})
        if (reinterpret_cast<uintptr_t>(p) % 16)
            return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: k, v, R_k, R_v and cache need to be 16-byte aligned", fn);
    return KVQ_OK;
}

kvq_status kvq_append_int4_launch(const char* fn, const AppendInt4& a, cudaStream_t st) {
    const int n_tok = a.n_tok, H_kv = a.H_kv;
    const int nsm = kvq_device_sm_count(), waves = (2 * H_kv + nsm - 1) / nsm;
    if ((int64_t)n_tok * H_kv < (int64_t)PREFILL_MIN * waves)
        return kvq_check_cuda(launch_pdl(append_int4_kernel, dim3(n_tok, H_kv, 2), dim3(512), 0, st, a), fn);
    const kvq_status sa = prefill_smem_once();
    if (sa != KVQ_OK) return sa;
    // One CTA per SM in all, each with a stride of its (head, side)'s tiles; a head's are
    // split between its sides so that the later of them ends soonest, in rounds of a tile
    // per worker (32K tokens, 8 heads, with read-back: 326 us for equal halves, 306 for 5 to 4,
    // 298 for 6 to 5).
    const int tiles = (n_tok + PF_M - 1) / PF_M, most = nsm / H_kv;
    auto rounds = [&](int ctas) { return (int)((tiles + (int64_t)ctas * PF_WORKERS - 1) / ((int64_t)ctas * PF_WORKERS)); };
    int nk = 1;
    int64_t best = INT64_MAX;
    float best_even = 0.f;
    for (int x = 1; x < most; ++x) {
        const int64_t cost = std::max((int64_t)PF_KEY_COST * rounds(x), (int64_t)PF_VALUE_COST * rounds(most - x));
        const float even = std::max((float)PF_KEY_COST / x, (float)PF_VALUE_COST / (most - x));
        if (cost < best || (cost == best && even < best_even)) {
            best = cost;
            best_even = even;
            nk = x;
        }
    }
    const int nv = std::min(tiles, std::max(1, most - nk));
    nk = std::min(tiles, nk);
    return kvq_check_cuda(launch_pdl(append_int4_prefill_kernel, dim3(nk + nv, H_kv), dim3(PF_WORKERS * 128), sizeof(PrefillSmem),
                                     st, a, nk),
                          fn);
}

extern "C" kvq_status kvq_append_int4(const void* k, const void* v, int n_tok, int H_kv, int d,
                                      const int32_t* slot_mapping, const float* mu_k, const float* R_k,
                                      const float* R_v, float clip, void* cache, int64_t num_pages,
                                      int32_t* err_count, void* stream) {
    AppendInt4 a = {};
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.k_stride = a.v_stride = (int64_t)H_kv * D;
    a.n_tok = n_tok;
    a.H_kv = H_kv;
    a.slot_mapping = slot_mapping;
    a.mu_k = mu_k;
    a.R_k = R_k;
    a.R_v = R_v;
    a.clip = clip;
    a.cache = static_cast<uint8_t*>(cache);
    a.num_pages = num_pages;
    a.err_count = err_count;
    const kvq_status st = kvq_append_int4_args("kvq_append_int4", a, d);
    if (st != KVQ_OK || n_tok == 0) return st;
    return kvq_append_int4_launch("kvq_append_int4 launch", a, static_cast<cudaStream_t>(stream));
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
