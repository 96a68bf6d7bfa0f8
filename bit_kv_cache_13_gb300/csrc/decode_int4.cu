// Fused packed-cache decode attention over the rotated INT4 cache, and the
// form that accumulates the attention weight each token drew.
//
//   q' = q R_k;  a_s = <q', K^_s> scale;  p = softmax(a);  o = (sum_s p_s V^_s) R_v^T
//
// Bound by the 160 bytes of packed cache per token-head, if the instructions
// that unpack them fit under the stream: one 12-warp CTA per SM, every warp
// streaming pages through a ring of its own (bulk copies, one mbarrier per unit
// of D4_U pages), all products on mma.sync m16n8k16 with the codes as operands.
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
//   softmax base 2, against the running maximum of each head; the maximum is
//           raised (and the accumulators rescaled) only when a logit exceeds it, which
//           one vote per unit decides.  Sums are fp32 of the unrounded p.
//   PV      rows = 16 channels, K = 16 tokens, columns = heads; the second operand is
//           fp16(fp16(p) * scale_{token, group}): two roundings of 2^-11 of a term, below
//           the output's bf16 rounding; p transposes from the QK layout by movmatrix.
//           Up to four heads fill the eight columns as (tokens 0..7, tokens 8..15) of
//           each head, which the end adds.  The mins are one more MMA.
//
// The work is split over the CTAs on the device, by the real page counts: the
// pages of all (sequence, KV head) units are laid end to end and every CTA takes
// an equal share, so a ragged batch or a short context in a long table stays
// balanced.  A CTA publishes one partial (m, l, o') per unit its share touches;
// the last to finish a unit (atomic ticket, no waiting) merges them by the
// log-sum-exp rule, rotates once by R_v^T and writes the output.  A unit with one
// partial is finished from shared memory.
#include <mutex>

#include "int4_common.cuh"

namespace kvq {

constexpr int D4_NW = 12;          // warps of a CTA, three per scheduler at 168 registers
constexpr int D4_THREADS = D4_NW * 32;
constexpr int D4_U = 2;            // pages per unit of a warp's ring
constexpr int D4_UNITS = 3;        // units in a ring
constexpr int D4_STAGES = D4_U * D4_UNITS;
constexpr int D4_MAX_SPLITS = 254;
constexpr int D4_MIN_PAGES = 16;   // pages a CTA takes at least when the split is automatic
constexpr int D4_SEG_PAGES = 50;   // what starting another unit costs a CTA, in pages streamed
constexpr float D4_NEG = -3e38f;   // running maximum before any token

__device__ __forceinline__ float d4_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Power of two that brings x into [2^14, 2^15) (1 for 0 and what is not
// finite; the exponent is held where neither it nor its inverse overflows).
__device__ __forceinline__ float d4_prescale(float x) {
    return x > 0.f && x < CUDART_INF_F ? ldexpf(1.f, max(-100, min(100, 14 - ilogbf(x)))) : 1.f;
}

// Transpose of an 8x8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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
    float* partials;   // [unit + CTA][G][PART_STRIDE]
    float* logits;     // [unit][16 max_pages][G], base 2 (weights form)
    float2* stats;     // [unit][G] (maximum, 1 / sum) (weights form)
    int automatic;     // the split is the kernel's choice (else the grid's)
};

template <int MAXG>
struct __align__(128) D4Smem {
    uint8_t ring[D4_NW][D4_STAGES][INT4_TILE];  // pages in flight; after a unit's last page, the warp's o' [G][D]
    uint64_t bar[D4_NW][D4_UNITS];
    int ntok[D4_NW][D4_STAGES];                 // valid tokens of the page in each slot
    float qin[MAXG][D];
    float q[MAXG][D];                           // q' * scale * log2(e); at the end the merged output
    float red[D4_NW][D];                        // partial sums of the rotation (3 parts a head) and of the merge
    float red2[MAXG == 8 ? 3 * MAXG - D4_NW : 1][D];
    uint4 bq[MAXG == 8 ? 8 : 1][32];            // eight heads: QK operands (high b0, b1, low b0, b1) per k step
    float gsum[MAXG][NGROUP];
    float sigma[MAXG], sigma_s[MAXG];           // power-of-two pre-scales of q' and S
    float m_part[D4_NW][MAXG], l_part[D4_NW][MAXG];
    float Mh[MAXG], Lh[MAXG];
    int64_t scan[D4_NW];
    int scan_max[D4_NW], scan_n[D4_NW];
    int64_t base0;
    int b0, is_last, dead;
};
static_assert(sizeof(D4Smem<4>) <= 227 * 1024 && sizeof(D4Smem<8>) <= 227 * 1024, "decode shared memory above 227 KB");
static_assert(8 * D * 4 <= D4_STAGES * INT4_TILE, "a warp's partial fits its ring");

// NT = 1: up to four query heads per KV head, NT = 2: up to eight.
template <int NT, bool WTS>
__global__ void __launch_bounds__(D4_THREADS, 1) decode_int4_kernel(const __grid_constant__ D4Args a) {
    constexpr int MAXG = 4 * NT;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    D4Smem<MAXG>& sm = *reinterpret_cast<D4Smem<MAXG>*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, t = lane & 3;
    const int G = a.G, cta = blockIdx.x;
    auto pages_of = [&](int b) {
        const int c = __ldg(a.context_lens + b);
        return c <= 0 ? 0 : min((int)(((int64_t)c + PAGE - 1) / PAGE), a.max_pages);
    };
    if (lane == 0) {
        for (int k = 0; k < D4_UNITS; ++k) mbar_init(&sm.bar[warp][k], 1);
        fence_mbar_init();
    }
    if (tid == 0) sm.dead = 0;
    griddep_wait();

    // ---- the split: pages of all sequences (a thread sums a run of them), the
    // CTAs that take part, and where this one's share begins
    int64_t V, g, g1;
    int Ceff;
    bool empties;
    {
        const int per = (a.B + D4_THREADS - 1) / D4_THREADS, s0 = min(a.B, tid * per), s1 = min(a.B, s0 + per);
        int64_t own = 0;
        int mx = 0, ne = 0;
        for (int b = s0; b < s1; ++b) {
            const int p = pages_of(b);
            own += p;
            mx = max(mx, p);
            ne += p > 0;
        }
        int64_t inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            ne += __shfl_xor_sync(0xffffffffu, ne, o);
        }
        if (lane == 31) {
            sm.scan[warp] = inc;
            sm.scan_max[warp] = mx;
            sm.scan_n[warp] = ne;
        }
        __syncthreads();
        int64_t P = 0, before = 0;
        mx = ne = 0;
#pragma unroll
        for (int w = 0; w < D4_NW; ++w) {
            if (w < warp) before += sm.scan[w];
            P += sm.scan[w];
            mx = max(mx, sm.scan_max[w]);
            ne += sm.scan_n[w];
        }
        empties = ne < a.B;
        V = P * a.H_kv;
        int64_t C = gridDim.x;
        if (a.automatic) {
            C = min(C, (V + D4_MIN_PAGES - 1) / D4_MIN_PAGES);
            // sequences of one length: a whole number of CTAs per unit, each in one
            // unit only, where that streams little more than equal shares would
            const int64_t units = (int64_t)ne * a.H_kv;
            if (units > 0 && units <= C && (int64_t)ne * mx == P) {
                const int64_t k = C / units;
                if ((mx + k - 1) / k <= V / C + D4_SEG_PAGES) C = units * k;
            }
        }
        if (C > V) C = V;
        Ceff = (int)C;
        g = g1 = 0;
        if (cta < Ceff) {
            g = (int64_t)cta * V / C;
            g1 = (int64_t)(cta + 1) * V / C;
            int64_t first = (before + inc - own) * a.H_kv;
            if (g >= first && g < first + own * a.H_kv) {
                int b = s0;
                for (; b < s1; ++b) {
                    const int64_t n = (int64_t)pages_of(b) * a.H_kv;
                    if (g < first + n) break;
                    first += n;
                }
                sm.b0 = b;
                sm.base0 = first;
            }
        }
    }
    if (empties)  // sequences without tokens: zeros
        for (int b = cta; b < a.B; b += gridDim.x)
            if (pages_of(b) == 0)
                for (int i = tid; i < a.H_q * D; i += D4_THREADS)
                    a.out[(size_t)b * a.H_q * D + i] = __float2bfloat16_rn(0.f);
    if (g >= g1) return;
    __syncthreads();

    auto cta_of = [&](int64_t x) { return (int)(((x + 1) * Ceff - 1) / V); };
    int b = sm.b0;
    int64_t base = sm.base0;  // first page of unit (b, 0)
    int np = pages_of(b);
    int h = (int)((g - base) / np);
    int kbase = 0;            // units this warp consumed in earlier segments
    while (true) {
        // ================ segment: pages [pa, pb) of unit (b, h)
        const int64_t ub = base + (int64_t)h * np;
        const int pa = (int)(g - ub), pb = (int)min((int64_t)np, g1 - ub);
        const size_t u = (size_t)b * a.H_kv + h;
        const int ctx = min(__ldg(a.context_lens + b), a.max_pages * PAGE);
        const int32_t* bt = a.block_table + (size_t)b * a.max_pages;
        const int count = sm.dead ? 0 : pb - pa;
        const int my_count = count > warp ? (count - warp + D4_NW - 1) / D4_NW : 0;
        const int n_units = (my_count + D4_U - 1) / D4_U;
        auto page_of = [&](int j) { return pa + warp + D4_NW * j; };
        int pid_first[D4_UNITS], pid_next = 0;
#pragma unroll
        for (int k = 0; k <= D4_UNITS; ++k) {
            const int j = D4_U * k + lane;
            const int pid = lane < D4_U && j < my_count ? __ldg(bt + page_of(j)) : 0;
            if (k < D4_UNITS)
                pid_first[k] = pid;
            else
                pid_next = pid;
        }
        // Lanes e < D4_U issue page e of unit k into ring group st and record its valid
        // tokens (0 for a page past the warp's or a bad id).
        auto issue_unit = [&](int k, int st, int pid) {
            uint64_t* bar = &sm.bar[warp][st];
            const int j = D4_U * k + lane;
            bool ok = false;
            if (lane < D4_U) {
                int n = 0;
                if (j < my_count) {
                    if (pid < 0 || (int64_t)pid >= a.num_pages) {
                        atomicOr(reinterpret_cast<uint32_t*>(a.ws), ERR_BAD_PAGE);
                    } else {
                        ok = true;
                        n = min(PAGE, ctx - page_of(j) * PAGE);
                    }
                }
                sm.ntok[warp][D4_U * st + lane] = n;
            }
            const uint32_t n_ok = __popc(__ballot_sync(0xffffffffu, ok));
            __syncwarp();  // the counts are ordered before lane 0's arrive
            if (lane == 0) {
                if (n_ok == 0)
                    mbar_arrive(bar);
                else
                    mbar_arrive_expect_tx(bar, n_ok * INT4_TILE);
            }
            __syncwarp();  // the expected bytes are set before any copy is issued
            if (ok)
                bulk_g2s_hint(sm.ring[warp][D4_U * st + lane], a.cache + ((size_t)pid * a.H_kv + h) * INT4_TILE, INT4_TILE,
                              bar, l2_policy_evict_first());
        };
        const int st0 = kbase % D4_UNITS;
        const uint32_t par0 = (kbase / D4_UNITS) & 1;
        int n_issued = 0;
#pragma unroll
        for (int k = 0; k < D4_UNITS; ++k)
            if (k < n_units) {
                issue_unit(k, st0 + k < D4_UNITS ? st0 + k : st0 + k - D4_UNITS, pid_first[k]);
                n_issued = k + 1;
            }

        // ---- q' = q R_k * scale * log2(e): thread (channel, third of the inputs)
        const __nv_bfloat16* qb = a.q + ((size_t)b * a.H_q + (size_t)h * G) * D;
        for (int i = tid; i < MAXG * D; i += D4_THREADS) sm.qin[i / D][i % D] = i < G * D ? __bfloat162float(qb[i]) : 0.f;
        auto red_row = [&](int part, int j) -> float* {
            const int x = part * MAXG + j;
            return x < D4_NW ? sm.red[x] : sm.red2[x - D4_NW];
        };
        {
            constexpr int PER = 44;  // 44 + 44 + 40 inputs, four at a time
            const int c = tid & (D - 1), part = tid >> 7, i0 = part * PER, i1 = min(D, i0 + PER);
            const float* R = a.Rk + (size_t)h * D * D + c;
            float rr[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) rr[i] = i0 + i < i1 ? __ldg(R + (size_t)(i0 + i) * D) : 0.f;
            __syncthreads();
            float acc[MAXG];
#pragma unroll
            for (int j = 0; j < MAXG; ++j) acc[j] = 0.f;
#pragma unroll
            for (int i = 0; i < PER; i += 4)
                if (i0 + i < i1) {
#pragma unroll
                    for (int j = 0; j < MAXG; ++j) {
                        const float4 x = *reinterpret_cast<const float4*>(&sm.qin[j][i0 + i]);
                        acc[j] = fmaf(x.x, rr[i], fmaf(x.y, rr[i + 1], fmaf(x.z, rr[i + 2], fmaf(x.w, rr[i + 3], acc[j]))));
                    }
                }
#pragma unroll
            for (int j = 0; j < MAXG; ++j) red_row(part, j)[c] = acc[j];
        }
        __syncthreads();
        // per head: sum the parts, the pre-scales (largest |q'| and |S| into [2^14, 2^15)) and the group sums
        if (warp < MAXG) {
            const int j = warp;
            float mx = 0.f, ms = 0.f, gs[NGROUP];
#pragma unroll
            for (int gg = 0; gg < NGROUP; ++gg) {
                const int c = 32 * gg + lane;
                const float x = (red_row(0, j)[c] + red_row(1, j)[c] + red_row(2, j)[c]) * a.scale_log2;
                sm.q[j][c] = x;
                mx = fmaxf(mx, fabsf(x));
                gs[gg] = x;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
                for (int gg = 0; gg < NGROUP; ++gg) gs[gg] += __shfl_xor_sync(0xffffffffu, gs[gg], o);
            }
#pragma unroll
            for (int gg = 0; gg < NGROUP; ++gg) ms = fmaxf(ms, fabsf(gs[gg]));
            if (lane == 0) {
                sm.sigma[j] = d4_prescale(mx);
                sm.sigma_s[j] = d4_prescale(ms);
#pragma unroll
                for (int gg = 0; gg < NGROUP; ++gg) sm.gsum[j][gg] = gs[gg];
            }
        }
        __syncthreads();
        // ---- QK operands.  K step 2 g + hs: b0 = channels 32 g + 8 t + 2 hs, + 4 (codes in
        // the low nibble), b1 = the channels after those (the next nibble, code * 16).
        auto q_frag = [&](int j, int s, int e, bool low) -> uint32_t {  // head j, k step s, register e
            const int c0 = 32 * (s >> 1) + 8 * t + 2 * (s & 1) + e;
            const float f = sm.sigma[j] * (e ? 0.0625f : 1.f);
            const float v0 = sm.q[j][c0] * f, v1 = sm.q[j][c0 + 4] * f;
            const float h0 = __half2float(__float2half_rn(v0)), h1 = __half2float(__float2half_rn(v1));
            return low ? pack_half2(v0 - h0, v1 - h1) : pack_half2(h0, h1);
        };
        auto s_frag = [&](int j, bool low) -> uint32_t {  // group sums 2 t, 2 t + 1 (t < 2)
            if (t >= 2) return 0u;
            const float v0 = sm.gsum[j][2 * t] * sm.sigma_s[j], v1 = sm.gsum[j][2 * t + 1] * sm.sigma_s[j];
            const float h0 = __half2float(__float2half_rn(v0)), h1 = __half2float(__float2half_rn(v1));
            return low ? pack_half2(v0 - h0, v1 - h1) : pack_half2(h0, h1);
        };
        uint32_t bq[NT == 1 ? 8 : 1][2], bs[2];
        float inv_q[NT], inv_s[NT];  // NT == 1: head t; NT == 2: heads 2 t, 2 t + 1
        if constexpr (NT == 1) {     // column r: head r / 2, high (r even) or low part
            const int j = r >> 1;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                bq[s][0] = q_frag(j, s, 0, r & 1);
                bq[s][1] = q_frag(j, s, 1, r & 1);
            }
            bs[0] = s_frag(j, r & 1);
            inv_q[0] = 16777216.f / sm.sigma[t];
            inv_s[0] = 1.f / sm.sigma_s[t];
        } else {                     // column r: head r
            if (warp < 8) sm.bq[warp][lane] = make_uint4(q_frag(r, warp, 0, false), q_frag(r, warp, 1, false),
                                                         q_frag(r, warp, 0, true), q_frag(r, warp, 1, true));
            bs[0] = s_frag(r, false);
            bs[1] = s_frag(r, true);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                inv_q[e] = 16777216.f / sm.sigma[2 * t + e];
                inv_s[e] = 1.f / sm.sigma_s[2 * t + e];
            }
            __syncthreads();
        }

        float oacc[8][4], cmin[4] = {0.f, 0.f, 0.f, 0.f}, mrun[NT], lsum[NT];
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[m][e] = 0.f;
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            mrun[e] = D4_NEG;
            lsum[e] = 0.f;
        }

        // base-2 logits of the page in ring slot: tokens r, r + 8 of head t (NT == 1), of heads 2 t, 2 t + 1 (NT == 2)
        auto qk_page = [&](int slot, float (&lg)[2][NT]) {
            const uint8_t* tile = sm.ring[warp][slot];
            const int n = sm.ntok[warp][slot];
            const uint4 ka = lds128(tile + O4_KC + 64 * r + 16 * t), kb = lds128(tile + O4_KC + 64 * (r + 8) + 16 * t);
            const uint2 sa = lds64(tile + O4_KM + 16 * r), sb = lds64(tile + O4_KM + 16 * (r + 8));
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
            const float2 fa0 = __half22float2(u32_as_h2(sa.x)), fa1 = __half22float2(u32_as_h2(sa.y));
            const float2 fb0 = __half22float2(u32_as_h2(sb.x)), fb1 = __half22float2(u32_as_h2(sb.y));
            const float fa[4] = {fa0.x, fa0.y, fa1.x, fa1.y}, fb[4] = {fb0.x, fb0.y, fb1.x, fb1.y};
            // min term: A column k = group k (the columns past 3 meet zeros)
            float cm[4] = {0.f, 0.f, 0.f, 0.f};
            {
                const uint32_t am[4] = {lds32(tile + O4_KM + 16 * r + 8 + 4 * (t & 1)),
                                        lds32(tile + O4_KM + 16 * (r + 8) + 8 + 4 * (t & 1)), 0u, 0u};
                mma_f16_16816(cm, am, bs[0], 0u);
                if constexpr (NT == 2) mma_f16_16816(cm, am, bs[1], 0u);
            }
            float xa[NT], xb[NT];
#pragma unroll
            for (int e = 0; e < NT; ++e) xa[e] = xb[e] = 0.f;
#pragma unroll
            for (int gg = 0; gg < NGROUP; ++gg) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int hs = 0; hs < 2; ++hs) {
                    const uint32_t A = hs ? wa[gg] >> 8 : wa[gg], Bw = hs ? wb[gg] >> 8 : wb[gg];
                    const uint32_t af[4] = {A & 0x000f000fu, Bw & 0x000f000fu, A & 0x00f000f0u, Bw & 0x00f000f0u};
                    if constexpr (NT == 1) {
                        mma_f16_16816(c, af, bq[2 * gg + hs][0], bq[2 * gg + hs][1]);
                    } else {
                        const uint4 f = sm.bq[2 * gg + hs][lane];
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
                lg[0][e] = r < n ? fmaf(xa[e], inv_q[e], ma * inv_s[e]) : -CUDART_INF_F;
                lg[1][e] = r + 8 < n ? fmaf(xb[e], inv_q[e], mb * inv_s[e]) : -CUDART_INF_F;
            }
        };

        auto pv_page = [&](int slot, const float (&p)[2][NT]) {
            const uint8_t* tile = sm.ring[warp][slot];
            uint32_t pb0, pb1;  // p in the operand's layout: tokens 2 t, 2 t + 1 and 2 t + 8, 2 t + 9
            uint32_t s0[4], s1[4];
            if constexpr (NT == 1) {
                // column r: head r / 2, tokens 0..7 (r even) or 8..15 (r odd); the other half is zero
                const uint32_t y = movmatrix(pack_half2(p[0][0], p[1][0]));
                pb0 = r & 1 ? 0u : y;
                pb1 = r & 1 ? y : 0u;
                const uint4 s = lds128(tile + O4_VS + 16 * (t + 4 * (r & 1)));
                s0[0] = s1[0] = s.x;
                s0[1] = s1[1] = s.y;
                s0[2] = s1[2] = s.z;
                s0[3] = s1[3] = s.w;
            } else {
                pb0 = movmatrix(pack_half2(p[0][0], p[0][1]));
                pb1 = movmatrix(pack_half2(p[1][0], p[1][1]));
                const uint4 sA = lds128(tile + O4_VS + 16 * t), sB = lds128(tile + O4_VS + 16 * (t + 4));
                s0[0] = sA.x;
                s0[1] = sA.y;
                s0[2] = sA.z;
                s0[3] = sA.w;
                s1[0] = sB.x;
                s1[1] = sB.y;
                s1[2] = sB.z;
                s1[3] = sB.w;
            }
            {   // min term: row r holds group r & 3
                const uint32_t am[4] = {lds32(tile + O4_VM + 16 * t + 4 * (r & 3)), 0u,
                                        lds32(tile + O4_VM + 16 * (t + 4) + 4 * (r & 3)), 0u};
                mma_f16_16816(cmin, am, pb0, pb1);
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
                    mma_f16_16816(oacc[2 * gg + hs], af, h0, h1);
                }
            }
        };

        // ---- the warp's pages
        int k_fail = -1, st = st0;
        uint32_t parity = par0;
        for (int k = 0; k < n_units; ++k) {
            const bool landed = mbar_wait_bounded(&sm.bar[warp][st], parity, WAIT_LIMIT_CYCLES);
            if (__any_sync(0xffffffffu, !landed)) {
                if (lane == 0) atomicOr(reinterpret_cast<uint32_t*>(a.ws), ERR_TIMEOUT);
                k_fail = k;
                break;
            }
            bool short_page = false;
#pragma unroll
            for (int e = 0; e < D4_U; ++e) short_page |= sm.ntok[warp][D4_U * st + e] < PAGE;
            if (short_page) {
                // slots past the context (or of no page) may hold any bytes, NaN too: their
                // value scales and mins are cleared, so p = 0 meets finite factors
                for (int x = lane; x < D4_U * 64; x += 32) {
                    const int e = x >> 6, w = x & 63, pair = (w & 31) >> 2, n = sm.ntok[warp][D4_U * st + e];
                    const uint32_t keep = (2 * pair < n ? 0x0000ffffu : 0u) | (2 * pair + 1 < n ? 0xffff0000u : 0u);
                    uint32_t* word = reinterpret_cast<uint32_t*>(sm.ring[warp][D4_U * st + e] + O4_VS) + w;
                    if (keep != 0xffffffffu) *word &= keep;
                }
                __syncwarp();
            }
            float lg[D4_U][2][NT];
#pragma unroll
            for (int e = 0; e < D4_U; ++e) qk_page(D4_U * st + e, lg[e]);
            if constexpr (WTS) {
#pragma unroll
                for (int e = 0; e < D4_U; ++e) {
                    const int j = D4_U * k + e;
                    if (j < my_count) {
                        float* row = a.logits + ((u * a.max_pages + page_of(j)) * PAGE + r) * G;
#pragma unroll
                        for (int x = 0; x < NT; ++x) {
                            const int hd = NT == 1 ? t : 2 * t + x;
                            if (hd < G) {
                                row[hd] = lg[e][0][x];
                                row[(size_t)8 * G + hd] = lg[e][1][x];
                            }
                        }
                    }
                }
            }
            float top[NT];
            bool grow = false;
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                top[x] = fmaxf(lg[0][0][x], lg[0][1][x]);
#pragma unroll
                for (int e = 1; e < D4_U; ++e) top[x] = fmaxf(top[x], fmaxf(lg[e][0][x], lg[e][1][x]));
                grow |= top[x] > mrun[x];
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 4));
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 8));
                    top[x] = fmaxf(fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 16)), mrun[x]);
                    const float c = d4_ex2(mrun[x] - top[x]);
                    mrun[x] = top[x];
                    lsum[x] *= c;
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
            }
#pragma unroll
            for (int e = 0; e < D4_U; ++e)
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    lg[e][0][x] = d4_ex2(lg[e][0][x] - mrun[x]);
                    lg[e][1][x] = d4_ex2(lg[e][1][x] - mrun[x]);
                    lsum[x] += lg[e][0][x] + lg[e][1][x];
                }
#pragma unroll
            for (int e = 0; e < D4_U; ++e) pv_page(D4_U * st + e, lg[e]);
            // hand the unit's slots back
            __syncwarp();
            if (k + D4_UNITS < n_units) {
                fence_proxy_async_smem();
                issue_unit(k + D4_UNITS, st, pid_next);
                n_issued = k + D4_UNITS + 1;
                const int j = D4_U * (k + D4_UNITS + 1) + lane;
                if (lane < D4_U && j < my_count) pid_next = __ldg(bt + page_of(j));
            }
            st = st + 1 == D4_UNITS ? 0 : st + 1;
            if (st == 0) parity ^= 1u;
        }
        if (k_fail >= 0 && lane == 0) {
            sm.dead = 1;
            // copies in flight land before the shared memory is reused
            for (int v = k_fail; v < n_issued; ++v)
                (void)mbar_wait_bounded(&sm.bar[warp][(kbase + v) % D4_UNITS], ((kbase + v) / D4_UNITS) & 1, 1000000LL);
        }
        __syncwarp();
        kbase += k_fail >= 0 ? n_issued : n_units;

        // ---- this warp's partial, in its own ring: channels 32 g + 4 r .. + 3 of its head(s)
        float* op = reinterpret_cast<float*>(sm.ring[warp][0]);
#pragma unroll
        for (int gg = 0; gg < NGROUP; ++gg) {
            if constexpr (NT == 1) {
                const float mt = __shfl_sync(0xffffffffu, cmin[0] + cmin[1], 4 * gg + t);
                *reinterpret_cast<float4*>(op + t * D + 32 * gg + 4 * r) =
                    make_float4(fmaf(oacc[2 * gg][0] + oacc[2 * gg][1], 16777216.f, mt),
                                fmaf(oacc[2 * gg][2] + oacc[2 * gg][3], 1048576.f, mt),
                                fmaf(oacc[2 * gg + 1][0] + oacc[2 * gg + 1][1], 16777216.f, mt),
                                fmaf(oacc[2 * gg + 1][2] + oacc[2 * gg + 1][3], 1048576.f, mt));
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float mt = __shfl_sync(0xffffffffu, cmin[x], 4 * gg + t);
                    *reinterpret_cast<float4*>(op + (2 * t + x) * D + 32 * gg + 4 * r) =
                        make_float4(fmaf(oacc[2 * gg][x], 16777216.f, mt), fmaf(oacc[2 * gg][2 + x], 1048576.f, mt),
                                    fmaf(oacc[2 * gg + 1][x], 16777216.f, mt), fmaf(oacc[2 * gg + 1][2 + x], 1048576.f, mt));
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
                sm.m_part[warp][hd] = mrun[x];
                sm.l_part[warp][hd] = l;
            }
        }
        __syncthreads();
        g = ub + pb;
        if (g >= g1) griddep_launch_dependents();

        // ---- merge the warps; publish, and finish the unit if this CTA is its last (or only) one
        const int c0 = cta_of(ub), n_part = cta_of(ub + np - 1) - c0 + 1;
        float* slot = a.partials + (u + cta) * (size_t)(G * PART_STRIDE);
        for (int i = tid; i < G * (D / 4); i += D4_THREADS) {
            const int j = i / (D / 4), c4 = 4 * (i % (D / 4));
            float M = D4_NEG, L = 0.f;
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < D4_NW; ++w) M = fmaxf(M, sm.m_part[w][j]);
#pragma unroll
            for (int w = 0; w < D4_NW; ++w) {
                const float f = d4_ex2(sm.m_part[w][j] - M);
                const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.ring[w][0]) + j * D + c4);
                L = fmaf(sm.l_part[w][j], f, L);
                O.x = fmaf(x.x, f, O.x);
                O.y = fmaf(x.y, f, O.y);
                O.z = fmaf(x.z, f, O.z);
                O.w = fmaf(x.w, f, O.w);
            }
            if (n_part == 1) {
                const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
                *reinterpret_cast<float4*>(&sm.q[j][c4]) = make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
                if (WTS && c4 == 0) a.stats[u * G + j] = make_float2(M, inv);
            } else {
                *reinterpret_cast<float4*>(slot + (size_t)j * PART_STRIDE + 4 + c4) = O;
                if (c4 == 0) *reinterpret_cast<float2*>(slot + (size_t)j * PART_STRIDE) = make_float2(M, L);
            }
        }
        fence_proxy_async_smem();  // the rings were written and read here: ordered before the next segment's copies
        __syncthreads();
        bool finish = true;
        if (n_part > 1) {
            int32_t* ticket = reinterpret_cast<int32_t*>(a.ws + WS_HEADER) + u;
            if (tid == 0) sm.is_last = atomic_add_acq_rel_gpu(ticket, 1) == n_part - 1;
            __syncthreads();
            finish = sm.is_last;
            if (finish) {
                if (tid == 0) *ticket = 0;
                // warp (part, head): partials part, part + P, ... with four channels a lane
                const int P = D4_NW / G, j = warp % G, part = warp / G;
                const float* ps = a.partials + (u + c0) * (size_t)(G * PART_STRIDE) + (size_t)j * PART_STRIDE;
                if (part < P) {
                    constexpr int CH = 8;
                    float M = D4_NEG, L = 0.f;
                    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int s0 = part; s0 < n_part; s0 += P * CH) {
                        float2 ml[CH];
                        float4 ov[CH];
#pragma unroll
                        for (int x = 0; x < CH; ++x) {
                            const int s = s0 + P * x;
                            const float* q = ps + (size_t)s * G * PART_STRIDE;
                            ml[x] = s < n_part ? __ldcg(reinterpret_cast<const float2*>(q)) : make_float2(D4_NEG, 0.f);
                            ov[x] = s < n_part ? __ldcg(reinterpret_cast<const float4*>(q + 4 + 4 * lane)) : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int x = 0; x < CH; ++x) {
                            const float Mn = fmaxf(M, ml[x].x), fo = d4_ex2(M - Mn), fn = d4_ex2(ml[x].x - Mn);
                            L = fmaf(L, fo, ml[x].y * fn);
                            O.x = fmaf(O.x, fo, ov[x].x * fn);
                            O.y = fmaf(O.y, fo, ov[x].y * fn);
                            O.z = fmaf(O.z, fo, ov[x].z * fn);
                            O.w = fmaf(O.w, fo, ov[x].w * fn);
                            M = Mn;
                        }
                    }
                    *reinterpret_cast<float4*>(&sm.red[warp][4 * lane]) = O;
                    if (lane == 0) {
                        sm.m_part[part][j] = M;
                        sm.l_part[part][j] = L;
                    }
                }
                __syncthreads();
                for (int i = tid; i < G * D; i += D4_THREADS) {
                    const int jj = i / D, c = i % D;
                    float M = D4_NEG, L = 0.f, O = 0.f;
                    for (int x = 0; x < P; ++x) M = fmaxf(M, sm.m_part[x][jj]);
                    for (int x = 0; x < P; ++x) {
                        const float f = d4_ex2(sm.m_part[x][jj] - M);
                        L = fmaf(sm.l_part[x][jj], f, L);
                        O = fmaf(sm.red[x * G + jj][c], f, O);
                    }
                    const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
                    sm.q[jj][c] = O * inv;
                    if (WTS && c == 0) a.stats[u * G + jj] = make_float2(M, inv);
                }
                __syncthreads();
            }
        }
        if (finish && warp < 8) {
            // out_i = sum_c o'_c R_v[i][c]: warp w takes rows 16 w .. + 15, a lane four
            // columns of each; a reduce-scatter leaves row lane % 16 in each lane
            const float* R = a.Rv + ((size_t)h * D + 16 * warp) * D + 4 * lane;
            float4 rr[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) rr[i] = __ldg(reinterpret_cast<const float4*>(R + (size_t)i * D));
            __nv_bfloat16* o = a.out + ((size_t)b * a.H_q + (size_t)h * G) * D + 16 * warp + lane;
            for (int j = 0; j < G; ++j) {
                const float4 x = *reinterpret_cast<const float4*>(&sm.q[j][4 * lane]);
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[i] = fmaf(x.x, rr[i].x, fmaf(x.y, rr[i].y, fmaf(x.z, rr[i].z, x.w * rr[i].w)));
                    v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
                }
#pragma unroll
                for (int off = 8; off >= 1; off >>= 1) {
                    const bool upper = lane & off;
#pragma unroll
                    for (int i = 0; i < off; ++i) {
                        const float send = upper ? v[i] : v[i + off], hold = upper ? v[i + off] : v[i];
                        v[i] = hold + __shfl_xor_sync(0xffffffffu, send, off);
                    }
                }
                if (lane < 16) o[(size_t)j * D] = __float2bfloat16_rn(v[0]);
            }
        }
        if (g >= g1) break;
        if (pb == np && ++h == a.H_kv) {
            h = 0;
            base += (int64_t)np * a.H_kv;
            do np = pages_of(++b);
            while (np == 0);
        }
        __syncthreads();  // the next segment reuses the scratch
    }
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

// CTAs of the decode: num_splits per (sequence, KV head) unit when given,
// else one per SM (the kernel uses as many of them as the pages deserve).
static int64_t d4_ctas(int B, int H_kv, int num_splits) {
    return num_splits > 0 ? (int64_t)num_splits * B * H_kv : kvq_device_sm_count();
}

struct D4Layout {
    size_t partials, stats, logits, total;
};
static D4Layout d4_layout(int B, int H_q, int H_kv, int max_pages, int64_t C, bool weights) {
    const size_t units = (size_t)B * H_kv, G = (size_t)(H_q / H_kv);
    D4Layout l;
    l.partials = WS_HEADER + tickets_bytes(B, H_kv);
    l.stats = align_up(l.partials + (units + (size_t)C) * G * PART_STRIDE * 4, 256);  // a slot per (unit + CTA)
    l.logits = align_up(l.stats + (weights ? units * G * 8 : 0), 256);
    l.total = l.logits + (weights ? units * (size_t)max_pages * PAGE * G * 4 : 0);
    return l;
}

extern "C" size_t kvq_int4_workspace_bytes(int B, int H_q, int H_kv, int max_pages_per_seq, int num_splits,
                                           int weights) {
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || max_pages_per_seq <= 0 || max_pages_per_seq >= (1 << 27) ||
        num_splits < 0 || num_splits > D4_MAX_SPLITS || B > 65535 || H_kv > 65535)
        return 0;
    return d4_layout(B, H_q, H_kv, max_pages_per_seq, d4_ctas(B, H_kv, num_splits), weights != 0).total;
}

// The shared memory opt-in is a per-device attribute of a kernel: set on the
// first call on each device only.
static kvq_status d4_smem_once(const void* fn, int bytes, int which) {
    static std::mutex mu;
    static bool done[64][4] = {};
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
    const int64_t C = d4_ctas(B, H_kv, num_splits);
    // (the kernel multiplies a CTA's index by the batch's pages in 64 bits)
    if (C > (1 << 22) || (int64_t)B * H_kv * max_pages > (int64_t(1) << 40))
        return kvq_set_error(KVQ_ERR_UNSUPPORTED, "%s: %lld CTAs above 2^22, or B * H_kv * max_pages above 2^40", fn, (long long)C);
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
    a.partials = reinterpret_cast<float*>(ws + lay.partials);
    a.stats = with_weights ? reinterpret_cast<float2*>(ws + lay.stats) : nullptr;
    a.logits = with_weights ? reinterpret_cast<float*>(ws + lay.logits) : nullptr;
    a.automatic = num_splits == 0;
    using Kern = decltype(&decode_int4_kernel<1, false>);
    static const Kern kerns[4] = {decode_int4_kernel<1, false>, decode_int4_kernel<1, true>, decode_int4_kernel<2, false>,
                                  decode_int4_kernel<2, true>};
    const int which = (G <= 4 ? 0 : 2) + (with_weights ? 1 : 0);
    const size_t smem = G <= 4 ? sizeof(D4Smem<4>) : sizeof(D4Smem<8>);
    kvq_status st = d4_smem_once((const void*)kerns[which], (int)smem, which);
    if (st != KVQ_OK) return st;
    st = kvq_check_cuda(launch_pdl(kerns[which], dim3((unsigned)C), dim3(D4_THREADS), smem, static_cast<cudaStream_t>(stream), a),
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
