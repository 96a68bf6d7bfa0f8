// Fused packed-cache decode attention over the rotated INT4 cache, and the
// form that accumulates the attention weight each token drew.
//
//   q' = q R_k;  a_s = <q', K^_s> scale;  p = softmax(a);  o = (sum_s p_s V^_s) R_v^T
//
// Bound by the 160 bytes of packed cache per token-head, if the instructions
// that unpack them fit under the stream (32 q / 8 KV heads, batch 1, 128K: 37 us, 4.5 TB/s;
// batch 8, 32K: 70.0 us, 4.8 TB/s; from 128K to 256K tokens another 25 us, 6.6 TB/s: the
// rest is the launch, the rotations, the merge).  One CTA of 12 warps per SM, every warp
// streaming pages through a ring of its own (bulk copies, one mbarrier per unit
// of one or two pages), all products on mma.sync m16n8k16 with the codes as operands.
//
//   codes   a 4-bit code masked out of its 16-bit half is an fp16 subnormal,
//           code * 2^-24 (low nibble) or 16 code * 2^-24 (next nibble): exact, one
//           AND for two codes, one shift for every four of them.
//   QK      rows = 16 tokens, K = channels, columns = heads.  a = sum_g scale_g
//           <q'_g, c_g> + sum_g min_g S_g with S_g the sum of q' over the group: two
//           MMAs per group and the scale applied to their fp32 result; the min term
//           is one more MMA over the four groups.  q' and S enter as an fp16 high and
//           low part (22 bits): for up to four heads the parts sit side by side in the
//           eight columns, for up to eight they are two MMAs into one accumulator.
//   softmax base 2, against the running maximum of each head, rounded up; the maximum is
//           raised (and the weights rescaled) only when a logit exceeds it, which
//           one vote per unit decides.  Sums are fp32 of the unrounded p.
//   PV      rows = 16 channels, K = 16 tokens, columns = heads; the second operand is
//           fp16(fp16(P) * scale_{token, group} / size): two roundings of 2^-11 of a term,
//           below the output's bf16 rounding.  A token's size is a power of two next
//           below the largest of its four scales and |mins|, and P = p * size relative to
//           a reference of its own, so that the largest P so far lies within 2^10 and 2^13.
//           So no operand overflows, and what fp16 cuts off below 2^-24 is 2^-29 of the
//           context's largest term, however small or large the weights are or the values
//           (6e-5 and up; smaller sizes count as that): a sink with small values, or none,
//           does not take the other tokens' digits.  P transposes from the QK layout by
//           movmatrix.  Up to four heads fill the eight columns as (tokens 0..7, tokens
//           8..15) of each head, which the end adds.  The mins are one more MMA.  A page's
//           products start from zero and are added in fp32, to nearest: an MMA cuts its
//           terms off toward zero, at 2^-25 of its accumulator, and the codes' and the
//           mins' sums, each of one sign, would drift apart (equal weights of 128K tokens
//           of values around zero in one CTA: 0.9 % of the output, 0.19 % so).
//
// Three kernels, chained by programmatic dependent launch so that each one's
// start overlaps the end of the one before:
//   1 rotate   q' of every (sequence, KV head), laid out as the MMA operand
//   2 stream   the cached pages; one partial (m, l, o') per CTA and unit
//   3 finish   merges a unit's partials by the log-sum-exp rule, rotates once by
//              R_v^T and writes the output; in the weights form more CTAs of the same
//              launch turn the logits that the stream left into token weights
// Rotating inside the streaming CTAs cost each (sequence, KV head) that a CTA
// touches about 7 us during which it streamed nothing (32 ragged sequences up to
// 4K, 8 KV heads: 166 us); where each CTA has one unit only, all three steps in one
// kernel are quicker instead (below, ONE).  The stream kernel's warps never wait for one another:
// each walks the CTA's units by itself, its ring running ahead into the next
// unit's pages; the last warp to leave a unit merges its warps' partials, which
// stand in ring slots of their own until then.
//
// The work is split over the CTAs on the device, by the real page counts: the
// pages of all (sequence, KV head) units are laid end to end and every CTA takes
// an equal share, so a ragged batch or a short context in a long table stays
// balanced.  With eight heads to a KV head the instructions bound it: 32 ragged
// sequences of up to 4K, 64 q / 8 KV heads, 53 us for 84 MB (12.5 at the copy rate).
#include <cstddef>
#include <mutex>

#include "int4_common.cuh"

namespace kvq {

// NW warps of a CTA (three per scheduler at 168 registers), U pages per unit of a
// warp's ring (one mbarrier phase, one refill), UNITS units in the ring.  Batch 8 at 32K,
// 32 q / 8 KV heads: 12 warps with three units 70.4 us, 8 warps with four 76.0; 128K, batch 1:
// 37.3 and 40.0.  (In a first form of the kernel, 128K: 12 warps with units of two pages
// 41.3 us, of one page 48.4, 16 warps with one page 49.4.)
template <int NT>
struct D4Cfg {
    static constexpr int NW = 12, U = 2, UNITS = 3;
};
constexpr int D4_MAX_SPLITS = 254;
constexpr int D4_MIN_PAGES = 24;   // pages per CTA below which an automatic split goes no further: a unit a warp
// What starting another unit costs a CTA, in pages streamed.  30 ragged sequences of up to
// 8000 tokens, 64 q / 8 KV heads: 84 us for 20, 69.7 for 40, 68.8 for 60, 70.8 for 110; 32 of
// up to 4000, 32 q heads: 49.4, 39.5, 39.5, 41.0.
constexpr int D4_SEG_PAGES = 60;
constexpr int D4_ONE_PAGES = 96;   // pages per CTA up to which a few sequences go without an even split
constexpr float D4_NEG = -3e38f;   // running maximum before any token
// PV weights P are at most 2^D4_PV_MOST (with scales below 4, products below 2^15); where one is
// above that, their reference moves, and the largest is 2^D4_PV_TOP or up to a bit less.
constexpr float D4_PV_MOST = 13.f, D4_PV_TOP = 11.f;
constexpr float D4_WHOLE = 12582912.f;  // 1.5 2^23: small numbers are rounded to whole ones by adding it
constexpr long long D4_SHORT_WAIT_CYCLES = 2000000LL;  // about a millisecond: a wait's limit under the test hook

__device__ __forceinline__ float d4_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Base-2 logarithm to 2^-22; -inf of 0.
__device__ __forceinline__ float d4_lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a + b, two fp32 sums in one instruction.
__device__ __forceinline__ float2 d4_add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Power of two that brings x into [2^14, 2^15) (1 for 0 and what is not
// finite; the exponent is held where neither it nor its inverse overflows).
__device__ __forceinline__ float d4_prescale(float x) {
    return x > 0.f && x < CUDART_INF_F ? ldexpf(1.f, max(-100, min(100, 14 - ilogbf(x)))) : 1.f;
}

// Transpose of an 8x8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// D = A(16x16 f16, row) * B(16x8 f16, col), fp32.
__device__ __forceinline__ void d4_mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two values' high fp16 parts, or what those leave of them.
__device__ __forceinline__ uint32_t d4_part(float v0, float v1, bool low) {
    const float h0 = __half2float(__float2half_rn(v0)), h1 = __half2float(__float2half_rn(v1));
    return low ? pack_half2(v0 - h0, v1 - h1) : pack_half2(h0, h1);
}

// The rotated queries of a unit as the stream kernel takes them: QK operands of
// the 8 k steps and 32 lanes (b0, b1 of the column's part; for NT == 2 the high
// part's, then the low part's), the min term's operand, and 2^24 / sigma and
// 1 / sigma_s of each head.
template <int NT>
struct __align__(16) D4Query {
    uint32_t bq[8][32][2 * NT];
    uint32_t bs[32][NT];
    float inv_q[4 * NT], inv_s[4 * NT];
};
static_assert(sizeof(D4Query<1>) % 16 == 0 && sizeof(D4Query<2>) % 16 == 0, "bulk copies take multiples of 16 bytes");

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
    void* query;       // D4Query [unit]
    int2* info;        // [unit] first CTA, partials
    float* partials;   // [unit + CTA][G][PART_STRIDE]
    float* logits;     // [unit][16 max_pages][G], base 2 (weights form)
    int automatic;     // the split is the kernel's choice (else the grid's)
    int drop;          // test hook: the first copy of CTA 0 is left out, and waits are short
    // weights form
    float* weights;
    int64_t wstride;
    float decay;
    int n_finish, chunks;
};

// ------------------------------------------------------------------ 1: rotate

// One CTA of 128 threads per KV head, group of 32 rotated channels and run of
// `per` sequences (a group is two K steps and one column of the min term).  Thread
// (channel, part) holds 32 rows of its column of R_k in registers.  The pre-scales
// come from the norm of q, which bounds every rotated value: |q'| sigma stays below
// 2^12 (fp16 ends at 2^16, so a matrix that is not quite a rotation has room) and
// |S| sigma_s, S a sum of 32, below 2^12 sqrt(32) / 8.  The kernel also has L2 fetch
// what the next two read first.
template <int NT>
__global__ void __launch_bounds__(128, 8) rotate_int4_kernel(const __grid_constant__ D4Args a, int per) {
    constexpr int MAXG = 4 * NT, PARTS = 4, ROWS = D / PARTS;
    __shared__ __align__(16) float qin[MAXG][D];
    __shared__ float red[PARTS][MAXG][32], qs[MAXG][32], gsum[MAXG], sigma[MAXG];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, t = lane & 3;
    const int h = blockIdx.x >> 2, g = blockIdx.x & 3, G = a.G;
    const float* R = a.Rk + (size_t)h * D * D + 32 * g + (size_t)ROWS * warp * D + lane;
    prefetch_l2(R - lane + (size_t)lane * D);
    prefetch_l2_keep(a.Rv + (size_t)h * D * D + 4096 * g + 32 * tid);
    griddep_wait();
    griddep_launch_dependents();  // (after the wait: what the next kernel reads early is complete)
    float rr[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) rr[i] = __ldg(R + (size_t)i * D);
    {
        const int64_t x = 128 * ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) + tid;  // lines of the tables
        if (x <= (a.B - 1) / 32) prefetch_l2(a.context_lens + 32 * x);
        if (x <= ((int64_t)a.B * a.max_pages - 1) / 32) prefetch_l2(a.block_table + 32 * x);
    }
    for (int b = blockIdx.y * per; b < min(a.B, (int)(blockIdx.y + 1) * per); ++b) {
        const __nv_bfloat16* qb = a.q + ((size_t)b * a.H_q + (size_t)h * G) * D;
        uint2 raw[NT];
#pragma unroll
        for (int e = 0; e < NT; ++e) {  // a warp per head (two for NT == 2): its values and their norm
            const int j = warp + 4 * e;
            raw[e] = j < G ? __ldg(reinterpret_cast<const uint2*>(qb + j * D) + lane) : make_uint2(0u, 0u);
        }
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            const int j = warp + 4 * e;
            const float4 x = make_float4(__uint_as_float(raw[e].x << 16), __uint_as_float(raw[e].x & 0xffff0000u),
                                         __uint_as_float(raw[e].y << 16), __uint_as_float(raw[e].y & 0xffff0000u));
            *reinterpret_cast<float4*>(&qin[j][4 * lane]) = x;
            float n2 = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w)));
#pragma unroll
            for (int o = 16; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
            if (lane == 0) sigma[j] = d4_prescale(sqrtf(n2) * fabsf(a.scale_log2) * 8.f);
        }
        __syncthreads();
        float acc[MAXG];
#pragma unroll
        for (int j = 0; j < MAXG; ++j) acc[j] = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS; i += 4)
#pragma unroll
            for (int j = 0; j < MAXG; ++j) {
                const float4 x = *reinterpret_cast<const float4*>(&qin[j][ROWS * warp + i]);
                acc[j] = fmaf(x.x, rr[i], fmaf(x.y, rr[i + 1], fmaf(x.z, rr[i + 2], fmaf(x.w, rr[i + 3], acc[j]))));
            }
#pragma unroll
        for (int j = 0; j < MAXG; ++j) red[warp][j][lane] = acc[j];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            const int j = warp + 4 * e;
            float x = ((red[0][j][lane] + red[1][j][lane]) + (red[2][j][lane] + red[3][j][lane])) * a.scale_log2;
            qs[j][lane] = x;
#pragma unroll
            for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0) gsum[j] = x;
        }
        __syncthreads();
        // K step 2 g + hs: b0 = channels 32 g + 8 t + 2 hs and + 4 (codes in the low nibble),
        // b1 = the channels after those (the next nibble: 16 times the code)
        auto q_frag = [&](int j, int e, bool low) {
            const int c0 = 8 * t + 2 * warp + e;
            const float f = sigma[j] * (e ? 0.0625f : 1.f);
            return d4_part(qs[j][c0] * f, qs[j][c0 + 4] * f, low);
        };
        D4Query<NT>& out = static_cast<D4Query<NT>*>(a.query)[(size_t)b * a.H_kv + h];
        if (warp < 2) {
            if constexpr (NT == 1)  // column r: head r / 2, high (r even) or low part
                *reinterpret_cast<uint2*>(out.bq[2 * g + warp][lane]) = make_uint2(q_frag(r >> 1, 0, r & 1), q_frag(r >> 1, 1, r & 1));
            else                    // column r: head r
                *reinterpret_cast<uint4*>(out.bq[2 * g + warp][lane]) =
                    make_uint4(q_frag(r, 0, false), q_frag(r, 1, false), q_frag(r, 0, true), q_frag(r, 1, true));
        } else if (warp == 2 && t == (g >> 1)) {
            // the min term's K index 2 t + e is group g: this CTA's half of lane (r, g / 2)
            const int j = NT == 1 ? r >> 1 : r;
            const float v = gsum[j] * sigma[j] * 0.125f, hi = __half2float(__float2half_rn(v));
            __half* bs = reinterpret_cast<__half*>(out.bs[lane]) + (g & 1);
            if constexpr (NT == 1) {
                bs[0] = __float2half_rn(r & 1 ? v - hi : hi);
            } else {
                bs[0] = __float2half_rn(hi);
                bs[2] = __float2half_rn(v - hi);
            }
        } else if (warp == 3 && g == 0) {
            if (t >= 2)
                for (int e = 0; e < NT; ++e) out.bs[lane][e] = 0u;
            if (lane < MAXG) {
                out.inv_q[lane] = 16777216.f / sigma[lane];
                out.inv_s[lane] = 8.f / sigma[lane];
            }
        }
        __syncthreads();  // sigma, qs and gsum are read above; the next round writes them
    }
}

// out_i = sum_c x_c R[i][c] for a warp's RW rows of R_v: a lane forms four columns
// of each, and a reduce-scatter leaves row lane % RW in each lane.
template <int RW>
__device__ __forceinline__ void d4_rotate_rows(float4 x, const float4 (&rr)[RW], int lane, __nv_bfloat16* out) {
    float v[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        v[i] = fmaf(x.x, rr[i].x, fmaf(x.y, rr[i].y, fmaf(x.z, rr[i].z, x.w * rr[i].w)));
#pragma unroll
        for (int off = 16; off >= RW; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    }
#pragma unroll
    for (int off = RW / 2; off >= 1; off >>= 1) {
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const float send = upper ? v[i] : v[i + off], hold = upper ? v[i + off] : v[i];
            v[i] = hold + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    if (lane < RW) out[lane] = __float2bfloat16_rn(v[0]);
}

// ------------------------------------------------------------------ 2: stream

__device__ __forceinline__ int d4_pages(const D4Args& a, int b) {
    const int c = __ldg(a.context_lens + b);
    return c <= 0 ? 0 : min((int)(((int64_t)c + PAGE - 1) / PAGE), a.max_pages);
}

// A CTA's walk over its share: pages [pa, pb) of unit (b, h), which has np (and
// `extra` without work after them), and `left` pages of the share after them.
struct D4Walk {
    int b, h, np, pa, pb, end, left;  // end: where the share leaves the unit, work-free pages counted
    // Takes [pa, ..) of the unit out of `share` pages; false if only work-free ones are left of it.
    __device__ __forceinline__ bool clip(int share, int extra) {
        end = (int)min((int64_t)np + extra, (int64_t)pa + share);
        left = share - (end - pa);
        pb = min(np, end);
        return pb > pa;
    }
    __device__ __forceinline__ void next(const D4Args& a, int extra) {  // needs left > 0
        if (++h == a.H_kv) {
            h = 0;
            do np = d4_pages(a, ++b);
            while (np == 0);
        }
        pa = 0;
        clip(left, extra);  // (a unit's first page is a real one)
    }
    // units of U pages that warp w of NW takes of the segment (its pages are dealt round-robin)
    template <int NW, int U>
    __device__ __forceinline__ int units(int w) const {
        const int n = pb - pa;
        const int mine = n > w ? (n - w + NW - 1) / NW : 0;
        return (mine + U - 1) / U;
    }
};

template <int NT>
struct __align__(128) D4Smem {
    static constexpr int NW = D4Cfg<NT>::NW, U = D4Cfg<NT>::U, UNITS = D4Cfg<NT>::UNITS;
    uint8_t ring[NW][U * UNITS][INT4_TILE];  // pages in flight; a unit's last slots keep the warp's o' [4 NT][D]
    D4Query<NT> query[2];                       // of segments s, s + 1
    uint64_t bar[NW][UNITS], qbar[2], free_bar[2];
    int ntok[NW][U * UNITS];                 // valid tokens of the page in each slot
    float m_part[2][NW][4 * NT], l_part[2][NW][4 * NT];
    int part_at[2][NW];                      // ring group that holds the warp's o', -1: no pages
    int arrived[2];
    int64_t scan[NW];
    int scan_max[NW], scan_n[NW];
    int64_t base0;
    int b0, is_last;
    // ONE: the query's rotation and the unit's end, in this kernel
    __align__(16) float qin[4 * NT][D];  // (these three are read as float4)
    __align__(16) float red[3][4 * NT][D];
    __align__(16) float qs[4 * NT][D];
    float gsum[4 * NT][NGROUP], sigma[4 * NT];
};
static_assert(offsetof(D4Smem<1>, qin) % 16 == 0 && offsetof(D4Smem<1>, red) % 16 == 0 && offsetof(D4Smem<1>, qs) % 16 == 0 &&
                  offsetof(D4Smem<2>, qin) % 16 == 0 && offsetof(D4Smem<2>, red) % 16 == 0 && offsetof(D4Smem<2>, qs) % 16 == 0 &&
                  offsetof(D4Smem<1>, query) % 16 == 0 && offsetof(D4Smem<2>, query) % 16 == 0 && offsetof(D4Smem<1>, bar) % 8 == 0 &&
                  offsetof(D4Smem<2>, bar) % 8 == 0,
              "wide accesses to shared memory are aligned");
static_assert(sizeof(D4Smem<1>) <= 227 * 1024 && sizeof(D4Smem<2>) <= 227 * 1024, "decode shared memory above 227 KB");
static_assert(4 * D * 4 <= D4Cfg<1>::U * INT4_TILE && 8 * D * 4 <= D4Cfg<2>::U * INT4_TILE, "a warp's partial fits one ring group");

// NT = 1: up to four query heads per KV head, NT = 2: up to eight.  ONE: the form
// for one or a few sequences, whole in this kernel: every CTA works on one unit, rotates
// its queries itself (before its first copies are out, so the rotation does not wait
// behind them) and the last CTA of a unit finishes it.
template <int NT, bool WTS, bool ONE>
__global__ void __launch_bounds__(D4Cfg<NT>::NW * 32, 1) decode_int4_kernel(const __grid_constant__ D4Args a) {
    constexpr int NW = D4Cfg<NT>::NW, U = D4Cfg<NT>::U, UNITS = D4Cfg<NT>::UNITS;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    D4Smem<NT>& sm = *reinterpret_cast<D4Smem<NT>*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, t = lane & 3;
    const int G = a.G, cta = blockIdx.x;
    if (lane == 0) {
        for (int k = 0; k < UNITS; ++k) mbar_init(&sm.bar[warp][k], 1);
        if (warp < 2) {
            mbar_init(&sm.qbar[warp], 1);
            mbar_init(&sm.free_bar[warp], 1);
            sm.arrived[warp] = 0;
        }
        fence_mbar_init();
    }
    __syncwarp();  // (a warp's ring is its own)

    // ---- the split: pages of all sequences (a thread sums a run of them), the
    // CTAs that take part, and where this one's share begins.  Context lengths,
    // block table and cache are read before the dependency wait: the rotate kernel
    // let this one start only after its own wait, when everything before it was done.
    int64_t V = 0, g0 = 0;
    int Ceff = 0, share = 0, part = 0, extra = 0;  // extra: pages without work after each unit's, for the cost of starting it
    D4Walk cs;  // what this warp consumes
    if constexpr (ONE) {
        griddep_wait();  // (no rotate kernel ran before)
        // a whole number of CTAs per unit, as many of them as its pages deserve
        const int most = gridDim.x / (a.B * a.H_kv), unit = cta / most;
        part = cta % most;
        cs.b = unit / a.H_kv;
        cs.h = unit % a.H_kv;
        cs.left = 0;
        cs.np = d4_pages(a, cs.b);
        if (cs.np == 0) {
            for (int i = tid; i < G * D && part == 0; i += NW * 32) a.out[(size_t)unit * G * D + i] = __float2bfloat16_rn(0.f);
            return;
        }
        Ceff = min(most, (cs.np + D4_MIN_PAGES - 1) / D4_MIN_PAGES);  // of the unit
        if (part >= Ceff) return;
        cs.pa = (int)((int64_t)part * cs.np / Ceff);
        cs.pb = cs.end = (int)((int64_t)(part + 1) * cs.np / Ceff);
    } else {
        const int per = (a.B + (NW * 32) - 1) / (NW * 32), s0 = min(a.B, tid * per), s1 = min(a.B, s0 + per);
        int64_t own = 0;
        int mx = 0, own_ne = 0;
        for (int b = s0; b < s1; ++b) {
            const int p = d4_pages(a, b);
            own += p;
            mx = max(mx, p);
            own_ne += p > 0;
        }
        int64_t inc = own;
        int inc_ne = own_ne;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
            const int y = __shfl_up_sync(0xffffffffu, inc_ne, o);
            if (lane >= o) {
                inc += x;
                inc_ne += y;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 31) {
            sm.scan[warp] = inc;
            sm.scan_max[warp] = mx;
            sm.scan_n[warp] = inc_ne;
        }
        __syncthreads();
        int64_t P = 0, before = 0;
        int ne = 0, before_ne = 0;
        mx = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) {
                before += sm.scan[w];
                before_ne += sm.scan_n[w];
            }
            P += sm.scan[w];
            mx = max(mx, sm.scan_max[w]);
            ne += sm.scan_n[w];
        }
        V = P * a.H_kv;
        int64_t C = gridDim.x;
        if (a.automatic) {
            const int64_t units = (int64_t)ne * a.H_kv;
            // (a CTA for each unit if there are as many: 19 sequences of one page in one CTA
            // took 88 us, a unit after the other)
            C = min(C, max((V + D4_MIN_PAGES - 1) / D4_MIN_PAGES, units));
            extra = D4_SEG_PAGES;
            // sequences of one length: a whole number of CTAs per unit, each in one
            // unit only, where that streams little more than equal shares would
            if (units > 0 && units <= C && (int64_t)ne * mx == P) {
                const int64_t k = C / units;
                if ((mx + k - 1) / k <= V / C + D4_SEG_PAGES) {
                    C = units * k;
                    extra = 0;
                }
            }
            own += (int64_t)own_ne * extra;
            before += (int64_t)before_ne * extra;
            inc += (int64_t)inc_ne * extra;
            V += units * extra;
        }
        if (C > V) C = V;
        Ceff = (int)C;
        if (cta >= Ceff) {
            griddep_wait();  // (a grid is complete only after the one before it)
            return;
        }
        g0 = (int64_t)cta * V / C;
        share = (int)((int64_t)(cta + 1) * V / C - g0);
        int64_t first = (before + inc - own) * a.H_kv;
        if (g0 >= first && g0 < first + own * a.H_kv) {
            int b = s0;
            for (; b < s1; ++b) {
                const int np = d4_pages(a, b);
                const int64_t n = (int64_t)(np ? np + extra : 0) * a.H_kv;
                if (g0 < first + n) break;
                first += n;
            }
            sm.b0 = b;
            sm.base0 = first;
        }
        __syncthreads();
    }
    if constexpr (!ONE) {
        cs.b = sm.b0;
        cs.np = d4_pages(a, cs.b);
        const int64_t in = g0 - sm.base0;
        cs.h = (int)(in / (cs.np + extra));
        cs.pa = (int)(in - (int64_t)cs.h * (cs.np + extra));
        if (!cs.clip(share, extra)) {
            if (cs.left == 0) {  // a share of work-free pages only
                griddep_wait();
                return;
            }
            cs.next(a, extra);
        }
    }

    // ONE: the head's R_k and queries are asked for before the pages
    constexpr int MAXG = 4 * NT, ROWS = ONE ? 44 : 1;  // 44 + 44 + 40 rows, four at a time
    float rr[ROWS], qv[ONE ? (MAXG * D + NW * 32 - 1) / (NW * 32) : 1];
    if constexpr (ONE) {
        const float* R = a.Rk + (size_t)cs.h * D * D + (tid & (D - 1));
        const int i0 = (tid >> 7) * ROWS;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) rr[i] = i0 + i < D ? __ldg(R + (size_t)(i0 + i) * D) : 0.f;
        const __nv_bfloat16* qb = a.q + ((size_t)cs.b * a.H_kv + cs.h) * G * D;
#pragma unroll
        for (int i = 0; i < (MAXG * D + NW * 32 - 1) / (NW * 32); ++i) {
            const int x = tid + i * NW * 32;
            qv[i] = x < G * D ? __bfloat162float(qb[x]) : 0.f;
        }
    }

    // ---- what it issues, up to UNITS units ahead, across segments.  Lane U x + e
    // of a batch holds page e of the batch's unit x: its id, KV head and valid tokens
    // (0: past the warp's pages).  The next batch's ids load while this one is issued.
    D4Walk is = cs;
    int ik = 0, in = is.units<NW, U>(warp), issued = 0, built = 0;
    constexpr int BATCH = 32 / U;
    auto build = [&](int& pid, int& hn) {  // the units after the first `built`
        pid = hn = 0;
        int x = 0;
        while (x < BATCH) {
            if (ik >= in) {
                if (is.left == 0) break;
                is.next(a, extra);
                ik = 0;
                in = is.units<NW, U>(warp);
                continue;
            }
            const int take = min(BATCH - x, in - ik), y = lane / U - x;
            const int page = is.pa + warp + NW * (U * (ik + y) + lane % U);
            if (y >= 0 && y < take && lane < U * BATCH && page < is.pb) {
                pid = __ldg(a.block_table + (size_t)is.b * a.max_pages + page);
                hn = is.h << 8 | (page + 1 < is.np ? PAGE : min(PAGE, __ldg(a.context_lens + is.b) - page * PAGE));
            }
            ik += take;
            x += take;
        }
        built += x;
    };
    int pid_n, hn_n;          // of the next batch: as loaded
    uint32_t tile_c, n_c;     // of this one: (page, KV head) tile, valid tokens (0: no page, or a bad id)
    uint32_t ok_mask = 0;     // lanes of this batch that hold a page
    bool any_bad = false;     // a bad id was seen: token counts are read back for every unit from then on
    auto turn = [&]() {       // the next batch becomes this one
        const bool page = hn_n & 255, ok = page && pid_n >= 0 && (int64_t)pid_n < a.num_pages;
        if (page && !ok) atomicOr(reinterpret_cast<uint32_t*>(a.ws), ERR_BAD_PAGE);
        any_bad |= __any_sync(0xffffffffu, page && !ok);
        tile_c = ok ? (uint32_t)pid_n * (uint32_t)a.H_kv + (uint32_t)(hn_n >> 8) : 0u;
        n_c = ok ? hn_n & 255 : 0;
        ok_mask = __ballot_sync(0xffffffffu, ok);
        build(pid_n, hn_n);
    };
    build(pid_n, hn_n);
    turn();
    const uint64_t policy = l2_policy_evict_first();
    int ist = 0, ix = 0;      // ring group and batch place of the next unit
    // Lanes e < U issue page e of the next unit.  (The copies may land before their
    // bytes are announced: the phase is open until lane 0 arrives.)
    auto issue_next = [&](bool drop) {
        if (ix == BATCH) {
            turn();
            ix = 0;
        }
        const int from = U * ix + lane % U;
        const uint32_t tile = __shfl_sync(0xffffffffu, tile_c, from), n = __shfl_sync(0xffffffffu, n_c, from);
        uint64_t* bar = &sm.bar[warp][ist];
        if (lane < U) {
            sm.ntok[warp][U * ist + lane] = (int)n;
            if (n && !(drop && lane == 0)) bulk_g2s_hint(sm.ring[warp][U * ist + lane], a.cache + (size_t)tile * INT4_TILE, INT4_TILE, bar, policy);
        }
        __syncwarp();  // the counts are ordered before the arrive
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(ok_mask >> (U * ix) & ((1u << U) - 1)) * INT4_TILE);
        ++issued;
        ++ix;
        ist = ist + 1 == UNITS ? 0 : ist + 1;
    };
    if (built > 0) issue_next(a.drop && tid < 32 && cta == 0);

    if constexpr (!ONE) {
        griddep_wait();  // the rotated queries are there
        griddep_launch_dependents();
    }
    auto fetch_query = [&](const D4Walk& w, int buf) {  // one thread
        mbar_arrive_expect_tx(&sm.qbar[buf], sizeof(D4Query<NT>));
        bulk_g2s(&sm.query[buf], static_cast<const D4Query<NT>*>(a.query) + ((size_t)w.b * a.H_kv + w.h), sizeof(D4Query<NT>),
                 &sm.qbar[buf]);
    };
    if (!ONE && tid == 0) {
        fetch_query(cs, 0);
        if (cs.left > 0) {
            D4Walk w = cs;
            w.next(a, extra);
            fetch_query(w, 1);
        }
    }
    // (the rest of the ring after the queries, which would queue behind it)
#pragma unroll 1
    while (issued < min(built, UNITS)) issue_next(false);
    if constexpr (ONE) {
        // q' = q R_k * scale * log2(e), as the rotate kernel has it, into query[0]
#pragma unroll
        for (int i = 0; i < (MAXG * D + NW * 32 - 1) / (NW * 32); ++i) {
            const int x = tid + i * NW * 32;
            if (x < MAXG * D) sm.qin[x / D][x % D] = qv[i];
        }
        __syncthreads();
        const int c = tid & (D - 1), part = tid >> 7, i0 = part * ROWS;
        float acc[MAXG];
#pragma unroll
        for (int j = 0; j < MAXG; ++j) acc[j] = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS; i += 4)
            if (i0 + i < D) {
#pragma unroll
                for (int j = 0; j < MAXG; ++j) {
                    const float4 x = *reinterpret_cast<const float4*>(&sm.qin[j][i0 + i]);
                    acc[j] = fmaf(x.x, rr[i], fmaf(x.y, rr[i + 1], fmaf(x.z, rr[i + 2], fmaf(x.w, rr[i + 3], acc[j]))));
                }
            }
#pragma unroll
        for (int j = 0; j < MAXG; ++j) sm.red[part][j][c] = acc[j];
        if (warp < MAXG) {
            const float4 x = *reinterpret_cast<const float4*>(&sm.qin[warp][4 * lane]);
            float n2 = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w)));
#pragma unroll
            for (int o = 16; o; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
            if (lane == 0) sm.sigma[warp] = d4_prescale(sqrtf(n2) * fabsf(a.scale_log2) * 8.f);
        }
        __syncthreads();
        for (int x = warp; x < MAXG * NGROUP; x += NW) {
            const int j = x / NGROUP, g = x % NGROUP, ch = 32 * g + lane;
            float y = ((sm.red[0][j][ch] + sm.red[1][j][ch]) + sm.red[2][j][ch]) * a.scale_log2;
            sm.qs[j][ch] = y;
#pragma unroll
            for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            if (lane == 0) sm.gsum[j][g] = y;
        }
        __syncthreads();
        D4Query<NT>& out = sm.query[0];
        auto q_frag = [&](int j, int e, bool low) {
            const int c0 = 32 * (warp >> 1) + 8 * t + 2 * (warp & 1) + e;
            const float f = sm.sigma[j] * (e ? 0.0625f : 1.f);
            return d4_part(sm.qs[j][c0] * f, sm.qs[j][c0 + 4] * f, low);
        };
        auto s_frag = [&](int j, bool low) {
            const float f = sm.sigma[j] * 0.125f;
            return t >= 2 ? 0u : d4_part(sm.gsum[j][2 * t] * f, sm.gsum[j][2 * t + 1] * f, low);
        };
        if (warp < 8) {
            if constexpr (NT == 1)
                *reinterpret_cast<uint2*>(out.bq[warp][lane]) = make_uint2(q_frag(r >> 1, 0, r & 1), q_frag(r >> 1, 1, r & 1));
            else
                *reinterpret_cast<uint4*>(out.bq[warp][lane]) =
                    make_uint4(q_frag(r, 0, false), q_frag(r, 1, false), q_frag(r, 0, true), q_frag(r, 1, true));
        } else if (warp == 8) {
            if constexpr (NT == 1)
                out.bs[lane][0] = s_frag(r >> 1, r & 1);
            else
                *reinterpret_cast<uint2*>(out.bs[lane]) = make_uint2(s_frag(r, false), s_frag(r, true));
        } else if (warp == 9 && lane < MAXG) {
            out.inv_q[lane] = 16777216.f / sm.sigma[lane];
            out.inv_s[lane] = 8.f / sm.sigma[lane];
        }
        __syncthreads();
    }

    bool dead = false;  // a wait of this warp ran out: it takes part without data
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
        const bool ok = mbar_wait_bounded(bar, parity, a.drop ? D4_SHORT_WAIT_CYCLES : WAIT_LIMIT_CYCLES);
        if (__any_sync(0xffffffffu, !ok)) {
            if (lane == 0) atomicOr(reinterpret_cast<uint32_t*>(a.ws), ERR_TIMEOUT);
            dead = true;
        }
    };
    int done = 0, st = 0;       // units consumed, the next one's ring group
    uint32_t parity = 0;        // and the parity of its phase
    int end1 = 0, end2 = 0;     // `done` at the end of the last segment, of the one before
    int freed = 0;              // units whose ring groups may be issued into again
    auto refill = [&]() {
#pragma unroll 1
        while (issued < min(built, freed + UNITS) && !dead) issue_next(false);
    };
    int s = 0;
    for (;; ++s) {
        // ================ segment s: pages [pa, pb) of unit (b, h)
        const size_t u = (size_t)cs.b * a.H_kv + cs.h;
        const int buf = s & 1;
        if (s >= 2) {
            // segment s - 2 is merged: its buffers, this one's queries (fetched by its last
            // warp) and the ring groups that held its partials
            wait(&sm.free_bar[buf], ((s - 2) >> 1) & 1);
            if (freed < end2) {
                freed = end2;
                fence_proxy_async_smem();  // (the partials were ordinary memory)
                refill();
            }
        }
        const int n_units = dead ? 0 : cs.units<NW, U>(warp);
        float oacc[8][4], cmin[4] = {0.f, 0.f, 0.f, 0.f}, mrun[NT], lsum[NT], vref[NT];  // whole numbers; vref: log2 of p * size where P is 1
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[m][e] = 0.f;
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            mrun[e] = D4_NEG;
            lsum[e] = 0.f;
            vref[e] = 0.f;
        }
        if (n_units > 0) {
            if constexpr (!ONE) wait(&sm.qbar[buf], (s >> 1) & 1);
            const D4Query<NT>& qf = sm.query[buf];
            uint32_t bq[NT == 1 ? 8 : 1][2], bs[2];
            float inv_q[NT], inv_s[NT];  // NT == 1: head t; NT == 2: heads 2 t, 2 t + 1
            if constexpr (NT == 1) {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint2 f = lds64(qf.bq[x][lane]);
                    bq[x][0] = f.x;
                    bq[x][1] = f.y;
                }
                bs[0] = bs[1] = qf.bs[lane][0];
                inv_q[0] = qf.inv_q[t];
                inv_s[0] = qf.inv_s[t];
            } else {
                const uint2 f = lds64(qf.bs[lane]);
                bs[0] = f.x;
                bs[1] = f.y;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    inv_q[e] = qf.inv_q[2 * t + e];
                    inv_s[e] = qf.inv_s[2 * t + e];
                }
            }

            // base-2 logits of the page in ring slot: tokens r, r + 8 of head t (NT == 1), of heads 2 t, 2 t + 1 (NT == 2)
            auto qk_page = [&](int slot, float (&lg)[2][NT]) {
                const uint8_t* tile = sm.ring[warp][slot];
                const uint4 ka = lds128(tile + O4_KC + 64 * r + 16 * t), kb = lds128(tile + O4_KC + 64 * (r + 8) + 16 * t);
                const uint2 sa = lds64(tile + O4_KM + 16 * r), sb = lds64(tile + O4_KM + 16 * (r + 8));
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
                const float2 fa0 = __half22float2(u32_as_h2(sa.x)), fa1 = __half22float2(u32_as_h2(sa.y));
                const float2 fb0 = __half22float2(u32_as_h2(sb.x)), fb1 = __half22float2(u32_as_h2(sb.y));
                const float fa[4] = {fa0.x, fa0.y, fa1.x, fa1.y}, fb[4] = {fb0.x, fb0.y, fb1.x, fb1.y};
                // min term: A column k = group k (the columns past 3 meet zeros)
                float cm[4];
                {
                    const uint32_t am[4] = {lds32(tile + O4_KM + 16 * r + 8 + 4 * (t & 1)),
                                            lds32(tile + O4_KM + 16 * (r + 8) + 8 + 4 * (t & 1)), 0u, 0u};
                    d4_mma0(cm, am, bs[0], 0u);
                    if constexpr (NT == 2) mma_f16_16816(cm, am, bs[1], 0u);
                }
                float xa[NT], xb[NT];
#pragma unroll
                for (int e = 0; e < NT; ++e) xa[e] = xb[e] = 0.f;
#pragma unroll
                for (int gg = 0; gg < NGROUP; ++gg) {
                    float c[4];
#pragma unroll
                    for (int hs = 0; hs < 2; ++hs) {
                        const uint32_t A = hs ? wa[gg] >> 8 : wa[gg], Bw = hs ? wb[gg] >> 8 : wb[gg];
                        const uint32_t af[4] = {A & 0x000f000fu, Bw & 0x000f000fu, A & 0x00f000f0u, Bw & 0x00f000f0u};
                        if constexpr (NT == 1) {
                            if (hs == 0)
                                d4_mma0(c, af, bq[2 * gg][0], bq[2 * gg][1]);
                            else
                                mma_f16_16816(c, af, bq[2 * gg + 1][0], bq[2 * gg + 1][1]);
                        } else {
                            const uint4 f = lds128(qf.bq[2 * gg + hs][lane]);
                            if (hs == 0)
                                d4_mma0(c, af, f.x, f.y);
                            else
                                mma_f16_16816(c, af, f.x, f.y);
                            mma_f16_16816(c, af, f.z, f.w);
                        }
                    }
                    if constexpr (NT == 1) {  // high + low part
                        xa[0] = fmaf(fa[gg], c[0] + c[1], xa[0]);
                        xb[0] = fmaf(fb[gg], c[2] + c[3], xb[0]);
                    } else {
                        xa[0] = fmaf(fa[gg], c[0], xa[0]);
                        xa[1] = fmaf(fa[gg], c[1], xa[1]);
                        xb[0] = fmaf(fb[gg], c[2], xb[0]);
                        xb[1] = fmaf(fb[gg], c[3], xb[1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < NT; ++e) {
                    const float ma = NT == 1 ? cm[0] + cm[1] : cm[e], mb = NT == 1 ? cm[2] + cm[3] : cm[2 + e];
                    lg[0][e] = fmaf(xa[e], inv_q[e], ma * inv_s[e]);
                    lg[1][e] = fmaf(xb[e], inv_q[e], mb * inv_s[e]);
                }
            };

            // Of the unit's two pages: log2 of the size of token lane & 15 of page lane >> 4, a whole
            // number, and the inverses of its slot pair's two sizes.  Sizes are powers of two within
            // 2^-14 and 2^14, so that both they and their inverses are fp16 numbers; of a token whose
            // values are 0 the logarithm is -inf.
            static_assert(U == 2, "half a warp a page");
            auto unit_sizes = [&](int group, float& logs, uint32_t& inv) {
                const uint8_t* at = sm.ring[warp][U * group + (lane >> 4)] + 8 * (lane & 15);  // groups 2 (lane & 1), + 1 of the pair
                const uint2 sc = lds64(at + O4_VS), mn = lds64(at + O4_VM);
                __half2 m = __hmax2(__hmax2(__habs2(u32_as_h2(sc.x)), __habs2(u32_as_h2(sc.y))),
                                    __hmax2(__habs2(u32_as_h2(mn.x)), __habs2(u32_as_h2(mn.y))));
                m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                const uint32_t size = h2_as_u32(__hmin2(__hmax2(m, u32_as_h2(0x04000400u)), u32_as_h2(0x74007400u))) & 0x7c007c00u;
                inv = 0x78007800u - size;
                const __half2 z = __hmin2(u32_as_h2(size), __hmul2(m, u32_as_h2(0x78007800u)));
                logs = (d4_lg2(__half2float(lane & 1 ? __high2half(z) : __low2half(z))) + D4_WHOLE) - D4_WHOLE;
            };

            auto pv_page = [&](int slot, uint32_t f, const uint32_t (&p)[NT]) {
                const uint8_t* tile = sm.ring[warp][slot];
                const bool odd = r & 1;
                uint32_t pb0, pb1;  // p in the operand's layout: tokens 2 t, 2 t + 1 and 2 t + 8, 2 t + 9
                uint32_t s0[4], s1[4];
                if constexpr (NT == 1) {
                    // column r: head r / 2, tokens 0..7 (r even) or 8..15 (r odd); the other half is zero
                    const uint32_t y = movmatrix(p[0]);
                    pb0 = odd ? 0u : y;
                    pb1 = odd ? y : 0u;
                    const uint4 sc = lds128(tile + O4_VS + 16 * (t + 4 * (r & 1)));
                    s0[0] = s1[0] = h2_as_u32(__hmul2(u32_as_h2(sc.x), u32_as_h2(f)));
                    s0[1] = s1[1] = h2_as_u32(__hmul2(u32_as_h2(sc.y), u32_as_h2(f)));
                    s0[2] = s1[2] = h2_as_u32(__hmul2(u32_as_h2(sc.z), u32_as_h2(f)));
                    s0[3] = s1[3] = h2_as_u32(__hmul2(u32_as_h2(sc.w), u32_as_h2(f)));
                } else {
                    pb0 = movmatrix(p[0]);
                    pb1 = movmatrix(p[1]);
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, f, 4);
                    const __half2 fa = u32_as_h2(odd ? other : f), fb = u32_as_h2(odd ? f : other);
                    const uint4 sA = lds128(tile + O4_VS + 16 * t), sB = lds128(tile + O4_VS + 16 * (t + 4));
                    s0[0] = h2_as_u32(__hmul2(u32_as_h2(sA.x), fa));
                    s0[1] = h2_as_u32(__hmul2(u32_as_h2(sA.y), fa));
                    s0[2] = h2_as_u32(__hmul2(u32_as_h2(sA.z), fa));
                    s0[3] = h2_as_u32(__hmul2(u32_as_h2(sA.w), fa));
                    s1[0] = h2_as_u32(__hmul2(u32_as_h2(sB.x), fb));
                    s1[1] = h2_as_u32(__hmul2(u32_as_h2(sB.y), fb));
                    s1[2] = h2_as_u32(__hmul2(u32_as_h2(sB.z), fb));
                    s1[3] = h2_as_u32(__hmul2(u32_as_h2(sB.w), fb));
                }
                {   // min term: row r holds group r / 2, tokens 0..7 (r even) or 8..15 (r odd)
                    const uint32_t m = h2_as_u32(__hmul2(u32_as_h2(lds32(tile + O4_VM + 16 * (t + 4 * (r & 1)) + 4 * (r >> 1))), u32_as_h2(f)));
                    const uint32_t am[4] = {odd ? 0u : m, 0u, odd ? m : 0u, 0u};
                    float d[4];
                    d4_mma0(d, am, pb0, pb1);
                    const float2 c = d4_add2(make_float2(cmin[0], cmin[1]), make_float2(d[0], d[1]));
                    cmin[0] = c.x;
                    cmin[1] = c.y;
                }
                const uint4 va = lds128(tile + O4_VC + 128 * t + 16 * r), vb = lds128(tile + O4_VC + 128 * (t + 4) + 16 * r);
                const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
                for (int gg = 0; gg < NGROUP; ++gg) {
                    const uint32_t h0 = h2_as_u32(__hmul2(u32_as_h2(pb0), u32_as_h2(s0[gg])));
                    const uint32_t h1 = h2_as_u32(__hmul2(u32_as_h2(pb1), u32_as_h2(s1[gg])));
#pragma unroll
                    for (int hs = 0; hs < 2; ++hs) {
                        const uint32_t A = hs ? wa[gg] >> 8 : wa[gg], Bw = hs ? wb[gg] >> 8 : wb[gg];
                        const uint32_t af[4] = {A & 0x000f000fu, A & 0x00f000f0u, Bw & 0x000f000fu, Bw & 0x00f000f0u};
                        float d[4];
                        d4_mma0(d, af, h0, h1);
                        float (&o)[4] = oacc[2 * gg + hs];
                        const float2 lo = d4_add2(make_float2(o[0], o[1]), make_float2(d[0], d[1])), hi = d4_add2(make_float2(o[2], o[3]), make_float2(d[2], d[3]));
                        o[0] = lo.x;
                        o[1] = lo.y;
                        o[2] = hi.x;
                        o[3] = hi.y;
                    }
                }
            };

            // Waits for the unit in ring group st and clears, where a page is short, what the
            // slots past the context (or of no page) hold: any bytes, NaN too; with zero value
            // scales and mins, p = 0 meets finite factors.  Returns the pages' token counts.
            // Only a warp's last unit of a segment can hold its end (`last`): the others are full,
            // unless a bad id was seen.
            struct Counts {
                int n[U];
            };
            auto wait_unit = [&](bool last) {
                Counts c;
#pragma unroll
                for (int e = 0; e < U; ++e) c.n[e] = PAGE;
                wait(&sm.bar[warp][st], parity);
                if (last || any_bad) {
                    int least = PAGE;
#pragma unroll
                    for (int e = 0; e < U; ++e) {
                        c.n[e] = sm.ntok[warp][U * st + e];
                        least = min(least, c.n[e]);
                    }
                    if (least < PAGE && !dead) {  // warp-uniform
                        for (int x = lane; x < U * 64; x += 32) {
                            const int e = x >> 6, w = x & 63, pair = (w & 31) >> 2, n = sm.ntok[warp][U * st + e];
                            const uint32_t keep = (2 * pair < n ? 0x0000ffffu : 0u) | (2 * pair + 1 < n ? 0xffff0000u : 0u);
                            uint32_t* word = reinterpret_cast<uint32_t*>(sm.ring[warp][U * st + e] + O4_VS) + w;
                            if (keep != 0xffffffffu) *word &= keep;
                        }
                        fence_proxy_async_smem();  // (written as ordinary memory: before the slots' next copies)
                        __syncwarp();
                    }
                }
                return c;
            };
            // Logits of page e of unit k (n valid tokens); the weights form stores them.
            auto logits = [&](int k, int slot, int e, int n, float (&lg)[2][NT]) {
                qk_page(slot, lg);
                if (n < PAGE) {  // warp-uniform
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        if (r >= n) lg[0][x] = -CUDART_INF_F;
                        if (r + 8 >= n) lg[1][x] = -CUDART_INF_F;
                    }
                }
                if constexpr (WTS) {
                    const int page = cs.pa + warp + NW * (U * k + e);
                    if (page < cs.pb) {
                        float* row = a.logits + ((u * a.max_pages + page) * PAGE + r) * G;
#pragma unroll
                        for (int x = 0; x < NT; ++x) {
                            const int hd = NT == 1 ? t : 2 * t + x;
                            if (hd < G) {
                                row[hd] = lg[0][x];
                                row[(size_t)8 * G + hd] = lg[1][x];
                            }
                        }
                    }
                }
            };
            // Rescales the value accumulators of this lane's head x.
            auto rescale = [&](int x, float c) {
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    oacc[m][x] *= c;
                    oacc[m][x + 2] *= c;
                    if (NT == 1) {
                        oacc[m][1] *= c;
                        oacc[m][3] *= c;
                    }
                }
                cmin[x] *= c;
                if (NT == 1) cmin[1] *= c;
            };
            // The softmax weights of a page's tokens (their sizes' logarithms in log_z) into the sums, and their PV
            // weights P: tokens r and r + 8 in one word, or (NT == 2) a word each of both heads.
            // Where a logit exceeds the running maximum or a P what it may be (one vote), the one
            // or the other reference is raised.
            auto softmax = [&](const float (&lg)[2][NT], float2 log_z, uint32_t (&p)[NT]) {
                float2 w[NT], P[NT];  // first their logarithms
                bool rare = false;
                auto relate = [&](int x) {  // (whole numbers first: what a reference moves by cancels exactly)
                    w[x] = d4_add2(make_float2(lg[0][x], lg[1][x]), make_float2(-mrun[x], -mrun[x]));
                    P[x] = d4_add2(w[x], d4_add2(log_z, make_float2(-vref[x], -vref[x])));
                };
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    relate(x);
                    rare |= fmaxf(lg[0][x], lg[1][x]) > mrun[x] || fmaxf(P[x].x, P[x].y) > D4_PV_MOST;
                }
                if (__any_sync(0xffffffffu, rare)) {
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        float top = fmaxf(lg[0][x], lg[1][x]), vtop = fmaxf(lg[0][x] + log_z.x, lg[1][x] + log_z.y);
#pragma unroll
                        for (int o = 4; o <= 16; o <<= 1) {
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, o));
                        }
                        top = fmaxf(ceilf(top), mrun[x]);
                        const float up = top - mrun[x];
                        lsum[x] *= d4_ex2(-up);
                        mrun[x] = top;
                        vref[x] -= up;  // (the values' sums stay)
                        vtop = ceilf((vtop - top) + fabsf(top) * 0x1p-22f);  // (with what its sum's rounding may have cost)
                        if (vtop - vref[x] > D4_PV_MOST) {
                            const float c = d4_ex2(vref[x] - (vtop - D4_PV_TOP));
                            vref[x] = vtop - D4_PV_TOP;
#pragma unroll
                            for (int m = 0; m < 8; ++m) {
                                oacc[m][x] *= c;
                                oacc[m][x + 2] *= c;
                                if (NT == 1) {
                                    oacc[m][1] *= c;
                                    oacc[m][3] *= c;
                                }
                            }
                            cmin[x] *= c;
                            if (NT == 1) cmin[1] *= c;
                        }
                        relate(x);
                    }
                }
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    P[x] = make_float2(d4_ex2(P[x].x), d4_ex2(P[x].y));
                    lsum[x] += d4_ex2(w[x].x) + d4_ex2(w[x].y);
                }
                if constexpr (NT == 1) {
                    p[0] = pack_half2(P[0].x, P[0].y);
                } else {
                    p[0] = pack_half2(P[0].x, P[1].x);
                    p[1] = pack_half2(P[0].y, P[1].y);
                }
            };

            // Pipelined by pages: the logits of the next page and the weighted sum of this
            // one share a block of code, so their latencies overlap.
            float lg[2][NT];
            uint32_t p[NT], invs = 0, f = 0, next = 0;  // f: 1 / size of tokens 2 t + 8 (r & 1) and the next, of the page whose weights p holds
            float logs = 0.f;
            auto page_logs = [&](int e) { return make_float2(__shfl_sync(0xffffffffu, logs, 16 * e + r), __shfl_sync(0xffffffffu, logs, 16 * e + r + 8)); };
            auto page_inv = [&](int e) { return __shfl_sync(0xffffffffu, invs, 16 * e + 2 * t + 8 * (r & 1)); };
            Counts nt = wait_unit(n_units == 1);
            if (!dead) {
                logits(0, U * st, 0, nt.n[0], lg);
                unit_sizes(st, logs, invs);
                f = page_inv(0);
            }
#pragma unroll 1
            for (int k = 0; k < n_units && !dead; ++k) {
                softmax(lg, page_logs(0), p);
#pragma unroll
                for (int e = 1; e < U; ++e) {
                    logits(k, U * st + e, e, nt.n[e], lg);
                    next = page_inv(e);
                    pv_page(U * st + e - 1, f, p);
                    f = next;
                    softmax(lg, page_logs(e), p);
                }
                ++done;
                const int last = U * st + U - 1;
                if (++st == UNITS) {
                    st = 0;
                    parity ^= 1u;
                }
                if (k + 1 == n_units) {
                    pv_page(last, f, p);
                    break;
                }
                nt = wait_unit(k + 2 == n_units);
                if (dead) break;
                logits(k + 1, U * st, 0, nt.n[0], lg);
                unit_sizes(st, logs, invs);
                next = page_inv(0);
                pv_page(last, f, p);
                f = next;
                __syncwarp();
                // hand the group back, and the ones that the last segment's partial held
                if (s > 0 && freed < end1) {
                    wait(&sm.free_bar[buf ^ 1], ((s - 1) >> 1) & 1);
                    fence_proxy_async_smem();  // (the partials were ordinary memory)
                }
                freed = done;
                refill();
            }
            __syncwarp();
        }
        if constexpr (WTS) {
            if (dead) {  // no logit of this warp's pages (what it wrote of them counts for nothing without its partial)
                for (int page = cs.pa + warp; page < cs.pb; page += NW)
                    for (int x = lane; x < PAGE * G; x += 32) a.logits[(u * a.max_pages + page) * PAGE * G + x] = -CUDART_INF_F;
            }
        }

        // ---- this warp's partial, in its last ring group: channels 32 g + 4 r .. + 3 of
        // its head(s)
        const bool has = n_units > 0 && !dead;
        const int at = st == 0 ? UNITS - 1 : st - 1;
        if (has) {
            float* op = reinterpret_cast<float*>(sm.ring[warp][U * at]);
            auto min_of = [&](float c, int g) { return __shfl_sync(0xffffffffu, c, 8 * g + t) + __shfl_sync(0xffffffffu, c, 8 * g + 4 + t); };
            // p size / P, and what the codes' places (2^-24, 2^-20) make of it
            float inv[NT], lo[NT], hi[NT];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                inv[x] = d4_ex2(vref[x]);
                lo[x] = 16777216.f * inv[x];
                hi[x] = 1048576.f * inv[x];
            }
#pragma unroll
            for (int gg = 0; gg < NGROUP; ++gg) {
                if constexpr (NT == 1) {
                    const float mt = min_of(cmin[0] + cmin[1], gg) * inv[0];
                    *reinterpret_cast<float4*>(op + t * D + 32 * gg + 4 * r) =
                        make_float4(fmaf(oacc[2 * gg][0] + oacc[2 * gg][1], lo[0], mt),
                                    fmaf(oacc[2 * gg][2] + oacc[2 * gg][3], hi[0], mt),
                                    fmaf(oacc[2 * gg + 1][0] + oacc[2 * gg + 1][1], lo[0], mt),
                                    fmaf(oacc[2 * gg + 1][2] + oacc[2 * gg + 1][3], hi[0], mt));
                } else {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float mt = min_of(cmin[x], gg) * inv[x];
                        *reinterpret_cast<float4*>(op + (2 * t + x) * D + 32 * gg + 4 * r) =
                            make_float4(fmaf(oacc[2 * gg][x], lo[x], mt), fmaf(oacc[2 * gg][2 + x], hi[x], mt),
                                        fmaf(oacc[2 * gg + 1][x], lo[x], mt), fmaf(oacc[2 * gg + 1][2 + x], hi[x], mt));
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            float l = lsum[x];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (r == 0) {
                const int hd = NT == 1 ? t : 2 * t + x;
                sm.m_part[buf][warp][hd] = has ? mrun[x] : D4_NEG;
                sm.l_part[buf][warp][hd] = has ? l : 0.f;
            }
        }
        if (lane == 0) sm.part_at[buf][warp] = has ? at : -1;
        if constexpr (ONE) {
            // ---- the whole CTA merges its warps; with more CTAs on the head it publishes, and
            // the last one merges those; then normalise, rotate by R_v^T, write
            __syncthreads();
            griddep_launch_dependents();
            const size_t step = (size_t)G * PART_STRIDE;
            float* slot = a.partials + (u + cta) * step;
            for (int i = tid; i < G * (D / 4); i += NW * 32) {
                const int j = i / (D / 4), c4 = 4 * (i % (D / 4));
                float M = D4_NEG, L = 0.f;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < NW; ++w) M = fmaxf(M, sm.m_part[0][w][j]);
#pragma unroll 4
                for (int w = 0; w < NW; ++w) {
                    const int at_w = sm.part_at[0][w];
                    const float f = d4_ex2(sm.m_part[0][w][j] - M);
                    if (at_w >= 0) {
                        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.ring[w][U * at_w]) + j * D + c4);
                        L = fmaf(sm.l_part[0][w][j], f, L);
                        O.x = fmaf(x.x, f, O.x);
                        O.y = fmaf(x.y, f, O.y);
                        O.z = fmaf(x.z, f, O.z);
                        O.w = fmaf(x.w, f, O.w);
                    }
                }
                if (Ceff == 1) {
                    const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
                    O = make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
                    *reinterpret_cast<float4*>(&sm.qs[j][c4]) = O;
                } else {
                    *reinterpret_cast<float4*>(slot + (size_t)j * PART_STRIDE + 4 + c4) = O;
                }
                if (c4 == 0) *reinterpret_cast<float2*>(slot + (size_t)j * PART_STRIDE) = make_float2(M, L);
            }
            if (WTS && tid == 0 && part == 0) a.info[u] = make_int2(cta, Ceff);
            __syncthreads();
            if (Ceff > 1) {
                int32_t* ticket = reinterpret_cast<int32_t*>(a.ws + WS_HEADER) + u;
                if (tid == 0) sm.is_last = atomic_add_acq_rel_gpu(ticket, 1) == Ceff - 1;
                __syncthreads();
                if (!sm.is_last) break;
                if (tid == 0) *ticket = 0;
                // warp (part, head): partials part, part + P, ..., four channels a lane
                const int P = NW / G, j = warp % G, p = warp / G;
                const float* ps = a.partials + (u + cta - part) * step + (size_t)j * PART_STRIDE;
                if (p < P) {
                    constexpr int CH = 8;
                    float M = D4_NEG, L = 0.f;
                    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int s0 = p; s0 < Ceff; s0 += P * CH) {
                        float2 ml[CH];
                        float4 ov[CH];
#pragma unroll
                        for (int x = 0; x < CH; ++x) {
                            const float* q = ps + (size_t)(s0 + P * x) * step;
                            const bool in_range = s0 + P * x < Ceff;
                            ml[x] = in_range ? __ldcg(reinterpret_cast<const float2*>(q)) : make_float2(D4_NEG, 0.f);
                            ov[x] = in_range ? __ldcg(reinterpret_cast<const float4*>(q + 4 + 4 * lane)) : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        float top = M;
#pragma unroll
                        for (int x = 0; x < CH; ++x) top = fmaxf(top, ml[x].x);
                        const float c = d4_ex2(M - top);
                        L *= c;
                        O = make_float4(O.x * c, O.y * c, O.z * c, O.w * c);
#pragma unroll
                        for (int x = 0; x < CH; ++x) {
                            const float f = d4_ex2(ml[x].x - top);
                            L = fmaf(ml[x].y, f, L);
                            O.x = fmaf(ov[x].x, f, O.x);
                            O.y = fmaf(ov[x].y, f, O.y);
                            O.z = fmaf(ov[x].z, f, O.z);
                            O.w = fmaf(ov[x].w, f, O.w);
                        }
                        M = top;
                    }
                    *reinterpret_cast<float4*>(&(&sm.red[0][0][0])[warp * D + 4 * lane]) = O;
                    if (lane == 0) {
                        sm.m_part[0][p][j] = M;
                        sm.l_part[0][p][j] = L;
                    }
                }
                __syncthreads();
                for (int i = tid; i < G * D; i += NW * 32) {
                    const int jj = i / D, c = i % D;
                    float M = D4_NEG, L = 0.f, O = 0.f;
                    for (int x = 0; x < P; ++x) M = fmaxf(M, sm.m_part[0][x][jj]);
                    for (int x = 0; x < P; ++x) {
                        const float f = d4_ex2(sm.m_part[0][x][jj] - M);
                        L = fmaf(sm.l_part[0][x][jj], f, L);
                        O = fmaf((&sm.red[0][0][0])[(x * G + jj) * D + c], f, O);
                    }
                    sm.qs[jj][c] = O * (L > 0.f ? 1.f / L : (L == L ? 0.f : L));
                }
                __syncthreads();
            }
            if (warp < 8) {
                const float* R = a.Rv + ((size_t)cs.h * D + 16 * warp) * D + 4 * lane;
                float4 rv[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) rv[i] = __ldg(reinterpret_cast<const float4*>(R + (size_t)i * D));
                __nv_bfloat16* o = a.out + u * G * D + 16 * warp;
#pragma unroll 1
                for (int jj = 0; jj < G; ++jj) d4_rotate_rows<16>(*reinterpret_cast<const float4*>(&sm.qs[jj][4 * lane]), rv, lane, o + (size_t)jj * D);
            }
            break;
        }
        end2 = end1;
        end1 = done;
        __syncwarp();
        int order = 0;
        fence_proxy_async_smem();
        if (lane == 0) {
            __threadfence_block();
            order = atomicAdd(&sm.arrived[buf], 1);
            __threadfence_block();
        }
        order = __shfl_sync(0xffffffffu, order, 0);
        if (order == NW - 1) {
            // ---- the last warp here merges its warps' partials in warp order and publishes
            __syncwarp();
            const int64_t ub = g0 + share - cs.left - cs.end;  // the unit's first page
            float* slot = a.partials + (u + cta) * (size_t)(G * PART_STRIDE);
            {
                // lane (row x0, head): the weights 2^(m_w - M) of warps x0, x0 + ROWS, ... in place
                // of m_w (0 without pages), and each head's M and L
                constexpr int MAXG = 4 * NT, ROWS = 32 / MAXG;
                const int j = lane % MAXG, x0 = lane / MAXG;
                float M = D4_NEG, L = 0.f;
#pragma unroll
                for (int w = x0; w < NW; w += ROWS) M = fmaxf(M, sm.m_part[buf][w][j]);
#pragma unroll
                for (int o = 16; o >= MAXG; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
                for (int w = x0; w < NW; w += ROWS) {
                    const float f = sm.part_at[buf][w] >= 0 ? d4_ex2(sm.m_part[buf][w][j] - M) : 0.f;
                    sm.m_part[buf][w][j] = f;
                    L = fmaf(sm.l_part[buf][w][j], f, L);
                }
#pragma unroll
                for (int o = 16; o >= MAXG; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
                if (lane < G) *reinterpret_cast<float2*>(slot + (size_t)lane * PART_STRIDE) = make_float2(M, L);
                __syncwarp();
            }
#pragma unroll 1
            for (int j = 0; j < G; ++j) {
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                constexpr int HALF = NW / 2;  // partials in flight
#pragma unroll
                for (int w0 = 0; w0 < NW; w0 += HALF) {
                    float4 x[HALF];
#pragma unroll
                    for (int w = 0; w < HALF; ++w) {
                        const int at_w = sm.part_at[buf][w0 + w];
                        x[w] = at_w >= 0 ? *reinterpret_cast<const float4*>(
                                               reinterpret_cast<const float*>(sm.ring[w0 + w][U * at_w]) + j * D + 4 * lane)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int w = 0; w < HALF; ++w) {
                        const float f = sm.m_part[buf][w0 + w][j];
                        O.x = fmaf(x[w].x, f, O.x);
                        O.y = fmaf(x[w].y, f, O.y);
                        O.z = fmaf(x[w].z, f, O.z);
                        O.w = fmaf(x[w].w, f, O.w);
                    }
                }
                *reinterpret_cast<float4*>(slot + (size_t)j * PART_STRIDE + 4 + 4 * lane) = O;
            }
            if (lane == 0) {
                auto cta_of = [&](int64_t x) { return (int)(((x + 1) * Ceff - 1) / V); };
                const int c0 = cta_of(ub);
                if (c0 == cta) a.info[u] = make_int2(c0, cta_of(ub + cs.np - 1) - c0 + 1);
                sm.arrived[buf] = 0;
            }
            __syncwarp();
            if (lane == 0) {
                // everyone is done with this segment's queries: fetch those of segment s + 2
                if (cs.left > 0) {
                    D4Walk w = cs;
                    w.next(a, extra);
                    if (w.left > 0) {
                        w.next(a, extra);
                        fence_proxy_async_smem();
                        fetch_query(w, buf);
                    }
                }
                mbar_arrive(&sm.free_bar[buf]);
            }
        }
        __syncwarp();
        if (cs.left == 0) break;
        cs.next(a, extra);
    }
    if (dead) {  // copies in flight land before the block ends, the last segments' queries too
        for (int v = done; v < issued; ++v)
            (void)mbar_wait_bounded(&sm.bar[warp][v % UNITS], (v / UNITS) & 1, 1000000LL);
        if constexpr (!ONE)
            for (int v = max(0, s - 1); v <= s; ++v) (void)mbar_wait_bounded(&sm.qbar[v & 1], (v >> 1) & 1, 1000000LL);
    }
}

// ------------------------------------------------------------------ 3: finish

// n_finish CTAs of 512 threads: RS of them per unit, D / RS rows of R_v each.
// They merge the unit's partials (warp = head and every P-th partial), normalise
// and rotate.  The others add weights: chunk x of a unit takes its tokens
// 512 x .. + 511 and every chunks * 512 on.
template <int RS, bool WTS>
__global__ void __launch_bounds__(512) finish_int4_kernel(const __grid_constant__ D4Args a) {
    constexpr int RW = D / RS / 16;  // rows of R_v a warp rotates
    __shared__ __align__(16) float part[16][D], o[8][D];
    __shared__ float Mh[8], inv[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.G;
    if (!WTS || (int)blockIdx.x < a.n_finish) {
        const size_t u = blockIdx.x / RS;
        const int b = (int)(u / a.H_kv), h = (int)(u % a.H_kv), row0 = (blockIdx.x % RS) * (D / RS) + RW * warp;
        // (R_v is read before the wait: the stream kernel started this one after its own wait)
        float4 rr[RW];
        const float* R = a.Rv + ((size_t)h * D + row0) * D + 4 * lane;
#pragma unroll
        for (int i = 0; i < RW; ++i) rr[i] = __ldg(reinterpret_cast<const float4*>(R + (size_t)i * D));
        const int pages = d4_pages(a, b);
        griddep_wait();
        griddep_launch_dependents();
        __nv_bfloat16* out = a.out + ((size_t)b * a.H_q + (size_t)h * G) * D + row0;
        if (pages == 0) {
            for (int i = lane; i < G * RW; i += 32) out[(size_t)(i / RW) * D + i % RW] = __float2bfloat16_rn(0.f);
            return;
        }
        const int2 info = __ldcg(a.info + u);
        const int P = 16 / G, j = warp % G, p = warp / G;
        if (p < P) {
            const float* ps = a.partials + (u + info.x) * (size_t)(G * PART_STRIDE) + (size_t)j * PART_STRIDE;
            const size_t step = (size_t)G * PART_STRIDE;
            // every warp of a head finds its M and L, a partial per lane; its own outputs are
            // partials p, p + P, ... (32 partials at a time, eight of its own in flight)
            float M = D4_NEG, L = 0.f;
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int base = 0; base < info.y; base += 32) {
                constexpr int CH = 8;
                float4 ov[CH];
                const int end = min(info.y, base + 32);
                const float2 ml = base + lane < end ? __ldcg(reinterpret_cast<const float2*>(ps + (base + lane) * step))
                                                    : make_float2(D4_NEG, 0.f);
                float top = M;
                for (int s0 = base + p; s0 < end; s0 += P * CH) {
#pragma unroll
                    for (int x = 0; x < CH; ++x)
                        ov[x] = s0 + P * x < end ? __ldcg(reinterpret_cast<const float4*>(ps + (s0 + P * x) * step + 4 + 4 * lane))
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                    if (s0 == base + p) {  // the running maximum, once the loads are out
                        top = fmaxf(M, ml.x);
#pragma unroll
                        for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                        const float c = d4_ex2(M - top);
                        O = make_float4(O.x * c, O.y * c, O.z * c, O.w * c);
                    }
                    const float f_own = d4_ex2(ml.x - top);
#pragma unroll
                    for (int x = 0; x < CH; ++x) {
                        const float f = __shfl_sync(0xffffffffu, f_own, (s0 + P * x - base) & 31);  // (past the end: times zeros)
                        O.x = fmaf(ov[x].x, f, O.x);
                        O.y = fmaf(ov[x].y, f, O.y);
                        O.z = fmaf(ov[x].z, f, O.z);
                        O.w = fmaf(ov[x].w, f, O.w);
                    }
                }
                if (base + p >= end) {  // no partial of its own here: only the maximum and the sum
                    top = fmaxf(M, ml.x);
#pragma unroll
                    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    const float c = d4_ex2(M - top);
                    O = make_float4(O.x * c, O.y * c, O.z * c, O.w * c);
                }
                float l = ml.y * d4_ex2(ml.x - top);
#pragma unroll
                for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
                L = fmaf(L, d4_ex2(M - top), l);
                M = top;
            }
            const float inv_l = L > 0.f ? 1.f / L : (L == L ? 0.f : L);  // no token: 0; NaN stays NaN
            *reinterpret_cast<float4*>(&part[warp][4 * lane]) = make_float4(O.x * inv_l, O.y * inv_l, O.z * inv_l, O.w * inv_l);
        }
        __syncthreads();
        if (tid < G * 32) {
            float4 x = *reinterpret_cast<const float4*>(&part[tid >> 5][4 * lane]);
            for (int y = 1; y < P; ++y) {
                const float4 z = *reinterpret_cast<const float4*>(&part[y * G + (tid >> 5)][4 * lane]);
                x = make_float4(x.x + z.x, x.y + z.y, x.z + z.z, x.w + z.w);
            }
            *reinterpret_cast<float4*>(&o[tid >> 5][4 * lane]) = x;
        }
        __syncthreads();
#pragma unroll 1
        for (int jj = 0; jj < G; ++jj) {
            d4_rotate_rows<RW>(*reinterpret_cast<const float4*>(&o[jj][4 * lane]), rr, lane, out + (size_t)jj * D);
        }
    } else {
        const int x = blockIdx.x - a.n_finish;
        const size_t u = x / a.chunks;
        const int chunk = x % a.chunks, b = (int)(u / a.H_kv);
        const int ctx = max(0, min(__ldg(a.context_lens + b), a.max_pages * PAGE));
        griddep_wait();
        griddep_launch_dependents();
        if (chunk * 512 >= ctx) return;
        // the unit's maximum and 1 / sum of each head
        const int2 info = __ldcg(a.info + u);
        if (warp < G) {
            const float* ps = a.partials + (u + info.x) * (size_t)(G * PART_STRIDE) + (size_t)warp * PART_STRIDE;
            float M = D4_NEG, L = 0.f;
            for (int s = lane; s < info.y; s += 32) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(ps + (size_t)s * G * PART_STRIDE));
                const float Mn = fmaxf(M, ml.x);
                L = fmaf(L, d4_ex2(M - Mn), ml.y * d4_ex2(ml.x - Mn));
                M = Mn;
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) {
                const float Mo = __shfl_xor_sync(0xffffffffu, M, off), Lo = __shfl_xor_sync(0xffffffffu, L, off);
                const float Mn = fmaxf(M, Mo);
                L = L * d4_ex2(M - Mn) + Lo * d4_ex2(Mo - Mn);
                M = Mn;
            }
            if (lane == 0) {
                Mh[warp] = M;
                inv[warp] = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
            }
        }
        __syncthreads();
        float* w = a.weights + (int64_t)u * a.wstride;
        const float* lg = a.logits + u * a.max_pages * PAGE * G;
        for (int64_t s = (int64_t)chunk * 512 + tid; s < ctx; s += (int64_t)a.chunks * 512) {
            float p = 0.f;
            auto add = [&](float z, int j) {
                // (a dropped token's logit is -inf: no weight, whatever the maximum)
                p += z == -CUDART_INF_F ? 0.f : d4_ex2(z - Mh[j]) * inv[j];
            };
            if (G % 4 == 0) {
                for (int j = 0; j < G; j += 4) {
                    const float4 z = __ldcg(reinterpret_cast<const float4*>(lg + (size_t)s * G + j));
                    add(z.x, j);
                    add(z.y, j + 1);
                    add(z.z, j + 2);
                    add(z.w, j + 3);
                }
            } else {
                for (int j = 0; j < G; ++j) add(__ldcg(lg + (size_t)s * G + j), j);
            }
            w[s] = fmaf(a.decay, w[s], p);
        }
    }
}

}  // namespace kvq

using namespace kvq;

// CTAs of the decode: num_splits per (sequence, KV head) unit when given,
// else one per SM (the kernel uses as many of them as the pages deserve).
static int64_t d4_ctas(int B, int H_kv, int num_splits) {
    return num_splits > 0 ? (int64_t)num_splits * B * H_kv : kvq_device_sm_count();
}

// (The tickets stand at one place whatever the shape, so that what a call of another
// shape left in the workspace is never taken for one.)
constexpr int D4_TICKETS = 1024;

struct D4Layout {
    size_t query, info, partials, logits, total;
};
static D4Layout d4_layout(int B, int H_q, int H_kv, int max_pages, int64_t C, bool weights) {
    const size_t units = (size_t)B * H_kv, G = (size_t)(H_q / H_kv);
    D4Layout l;
    l.query = WS_HEADER + D4_TICKETS * 4;
    l.info = align_up(l.query + units * (G <= 4 ? sizeof(D4Query<1>) : sizeof(D4Query<2>)), 256);
    l.partials = align_up(l.info + units * sizeof(int2), 256);
    l.logits = align_up(l.partials + (units + (size_t)C) * G * PART_STRIDE * 4, 256);  // a slot per (unit + CTA)
    l.total = l.logits + (weights ? units * (size_t)max_pages * PAGE * G * 4 : 0);
    return l;
}

// What the arguments that the workspace depends on are refused for (null: nothing).
static const char* d4_refusal(int B, int H_q, int H_kv, int max_pages, int num_splits, kvq_status& st) {
    st = KVQ_ERR_INVALID_ARG;
    if (B <= 0 || H_kv <= 0 || H_q <= 0 || H_q % H_kv || max_pages <= 0 || num_splits < 0) return "sizes";
    if (num_splits > D4_MAX_SPLITS) return "num_splits above 254";
    st = KVQ_ERR_UNSUPPORTED;
    if (H_q / H_kv > 8) return "GQA group above 8";
    if (B > 65535 || H_kv > 65535) return "B or H_kv above 65535";
    if (max_pages >= (1 << 27)) return "max_pages_per_seq not below 2^27";
    const int64_t units = (int64_t)B * H_kv;
    if (units > (1 << 24)) return "B * H_kv above 2^24";
    // (a CTA's index times the batch's pages stays within 64 bits, a CTA's share within 32)
    if (units * max_pages > (int64_t(1) << 36)) return "B * H_kv * max_pages_per_seq above 2^36";
    if (units * num_splits > (1 << 22)) return "more than 2^22 CTAs";
    st = KVQ_OK;
    return nullptr;
}

extern "C" size_t kvq_int4_workspace_bytes(int B, int H_q, int H_kv, int max_pages_per_seq, int num_splits,
                                           int weights) {
    kvq_status st;
    if (d4_refusal(B, H_q, H_kv, max_pages_per_seq, num_splits, st)) return 0;
    return d4_layout(B, H_q, H_kv, max_pages_per_seq, d4_ctas(B, H_kv, num_splits), weights != 0).total;
}

// The shared memory opt-in is a per-device attribute of a kernel: set on the
// first call on each device only.
static kvq_status d4_smem_once(const void* fn, int bytes, int which) {
    static std::mutex mu;
    static bool done[64][8] = {};
    int dev = 0;
    kvq_status st = kvq_check_cuda(cudaGetDevice(&dev), "kvq_decode_attn_int4: cudaGetDevice");
    if (st != KVQ_OK) return st;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && done[dev][which]) return KVQ_OK;
    st = kvq_check_cuda(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes),
                        "kvq_decode_attn_int4 smem attribute");
    if (st == KVQ_OK && dev >= 0 && dev < 64) done[dev][which] = true;
    return st;
}

static kvq_status decode_int4(const char* fn, const void* q, int B, int H_q, int H_kv, int d, const void* cache,
                              int64_t num_pages, const int32_t* block_table, int max_pages,
                              const int32_t* context_lens, const float* R_k, const float* R_v, float scale, void* out,
                              bool with_weights, float* weights, int64_t weights_stride, float decay, void* workspace,
                              size_t workspace_bytes, int num_splits, void* stream) {
    if (d != D) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: d=%d (only 128)", fn, d);
    kvq_status st;
    if (const char* why = d4_refusal(B, H_q, H_kv, max_pages, num_splits, st))
        return kvq_set_error(st, "%s: %s (B=%d H_q=%d H_kv=%d max_pages=%d splits=%d)", fn, why, B, H_q, H_kv, max_pages,
                             num_splits);
    if (num_pages <= 0) return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: num_pages=%lld", fn, (long long)num_pages);
    const int G = H_q / H_kv;
    if (!q || !cache || !block_table || !context_lens || !R_k || !R_v || !out || !workspace || (with_weights && !weights))
        return kvq_set_error(KVQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (num_pages > (int64_t(1) << 32) / H_kv) return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: num_pages * H_kv above 2^32", fn);
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
    const int64_t C = d4_ctas(B, H_kv, num_splits);
    const D4Layout lay = d4_layout(B, H_q, H_kv, max_pages, C, with_weights);
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
    a.query = ws + lay.query;
    a.info = reinterpret_cast<int2*>(ws + lay.info);
    a.partials = reinterpret_cast<float*>(ws + lay.partials);
    a.logits = with_weights ? reinterpret_cast<float*>(ws + lay.logits) : nullptr;
    a.automatic = num_splits == 0;
    a.drop = kvq_take_drop_next_copy();
    a.weights = weights;
    a.wstride = weights_stride;
    a.decay = decay;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int nsm = kvq_device_sm_count();
    const int64_t units = (int64_t)B * H_kv;
    // A few units: one kernel (in the weights form, and the weights' one), whose CTAs have one
    // unit each.  Lengths differ, so of several sequences none may have more than
    // D4_ONE_PAGES pages for each of its CTAs.  8 sequences of 300 tokens, 8 KV heads: 9.3 us
    // against 12.8 in three kernels, 16 of 1500 14.2 against 20.2; 3 of up to 8000 (84 pages a
    // CTA) 16.5 against 14.7.  In the weights form, where the third kernel runs anyway and
    // would have merged the partials, only up to two CTAs per unit (8 of 700 tokens 14.4
    // against 15.5 us, but 4 of up to 1959 with 4 heads 14.4 against 13.7) and for a single
    // sequence (2048 tokens: 14.3 against 13.6 us in a graph, but one launch fewer to pay for
    // on the host).
    const int per_unit = (int)(nsm / units);
    const bool small = max_pages <= (int64_t)D4_ONE_PAGES * per_unit;
    const bool one = num_splits == 0 && per_unit >= 1 && units <= D4_TICKETS &&
                     ((small && (!with_weights || per_unit <= 2)) || (B == 1 && per_unit >= 4));
    if (!one) {
        // 1: one sequence a CTA, up to eight CTAs per SM
        const int per = (int)((4 * units + 8 * nsm - 1) / (8 * nsm));
        st = kvq_check_cuda(launch_pdl(G <= 4 ? rotate_int4_kernel<1> : rotate_int4_kernel<2>,
                                       dim3(4 * H_kv, (B + per - 1) / per), dim3(128), 0, cs, a, per),
                            "kvq_decode_attn_int4 rotate launch");
        if (st != KVQ_OK) return st;
    }
    // 2
    using Kern = decltype(&decode_int4_kernel<1, false, false>);
    static const Kern kerns[8] = {decode_int4_kernel<1, false, false>, decode_int4_kernel<1, true, false>,
                                  decode_int4_kernel<2, false, false>, decode_int4_kernel<2, true, false>,
                                  decode_int4_kernel<1, false, true>,  decode_int4_kernel<1, true, true>,
                                  decode_int4_kernel<2, false, true>,  decode_int4_kernel<2, true, true>};
    const int which = (G <= 4 ? 0 : 2) + (with_weights ? 1 : 0) + (one ? 4 : 0);
    const size_t smem = G <= 4 ? sizeof(D4Smem<1>) : sizeof(D4Smem<2>);
    st = d4_smem_once((const void*)kerns[which], (int)smem, which);
    if (st != KVQ_OK) return st;
    st = kvq_check_cuda(launch_pdl(kerns[which], dim3(one ? (unsigned)(units * per_unit) : (unsigned)C), dim3(32 * (G <= 4 ? D4Cfg<1>::NW : D4Cfg<2>::NW)), smem, cs, a),
                        "kvq_decode_attn_int4 launch");
    if (st != KVQ_OK || (one && !with_weights)) return st;
    // 3: few units are finished by four CTAs each (a quarter of R_v each), and
    // about two CTAs per SM share the weights
    const bool few = units * 4 <= nsm;
    a.n_finish = one ? 0 : (int)(units * (few ? 4 : 1));
    a.chunks = 0;
    if (with_weights) {
        const int64_t blocks = ((int64_t)max_pages * PAGE + 511) / 512, most = (2 * nsm + units - 1) / units;
        a.chunks = (int)(blocks < most ? blocks : most);
    }
    const dim3 grid((unsigned)(a.n_finish + units * a.chunks));
    st = kvq_check_cuda(launch_pdl(with_weights ? (few ? finish_int4_kernel<4, true> : finish_int4_kernel<1, true>)
                                                : (few ? finish_int4_kernel<4, false> : finish_int4_kernel<1, false>),
                                   grid, dim3(512), 0, cs, a),
                        "kvq_decode_attn_int4 finish launch");
    return st;
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
