// Attention of each sequence's last tokens over the rotated INT4 cache: a piece of a
// prompt, drafted tokens, or a whole prompt, causal among themselves, with an optional
// sliding window and sinks.
//
//   q' = q R_k;  a_t = <q', K^_t> scale over the tokens that the query's position sees;
//   o = (sum_t softmax(a)_t V^_t) R_v^T
//
// Three kernels, chained by programmatic dependent launch:
//   1 rotate   q' of every row (a token and one of its heads) as fp16, and the plan: the
//              row blocks with the tiles of tokens that they see
//   2 stream   a persistent CTA per SM takes an equal share of all blocks' tiles; the
//              products on tcgen05, the cache unpacked to fp16 in shared memory on the way
//   3 finish   merges the shares' partial sums, normalises, rotates by R_v^T
#include <algorithm>
#include <cstddef>
#include <mutex>

#include "int4_common.cuh"

namespace kvq {

constexpr int CK_ROWS = 256;       // most rows of a block: two row tiles of 128
constexpr int CK_ROW_TILE = 128;
constexpr int CK_PAGES = 4, CK_TILE = CK_PAGES * PAGE;  // pages and cached tokens of a tile
// What starting a block costs, in tiles of one row tile: its queries' way in, a pipeline filled and drained, its sums' way
// out.  A 4K prompt: 312 us for 8, 278 for 11, 256 for 14, 252 for 18, 258 for 24; 8 x 5 tokens at 32K, in blocks of one row
// tile: 191 us for 4 and 6, 192 for 9.
constexpr int CK_UNIT_COST = 18, CK_UNIT_COST_FEW = 6;
// The least share worth a CTA, in the same units: the finish merges a block's shares one after the other.  32 q / 8 KV heads,
// 5 tokens of 2000: 58 us for 1, 36 for 6, 34 for 12 and 20, 49 for 45; 5 of 500: 29, 26, 29, 33, 44; 64 of 1000, in blocks
// of two row tiles: 75 for 1, 45 for 12 and 20, 54 for 45; 64 of 4000: 75 for 12, 63 for 20, 62 for 45.
constexpr int CK_LEAST_SHARE = 20, CK_LEAST_SHARE_FEW = 12;
// Most tiles of a block that are summed in tensor memory at a time: a product cuts its sum off below fp32, by 2^-23.6 of it on
// the average, so that the 4 * 16384 of a million tokens of equal weight took 0.3 % off.  What a CTA has of a block beyond
// that is a run of its own, added in fp32 to the partial before it (1024 tiles, 64K tokens: at most 2^-11).
constexpr int CK_RUN = 1024;
constexpr float CK_NEG = -3e38f;   // reference of a row before it sees a token
// A token counts in the output by its weight times the size of its values: the power of two of 8 |scale| + |min| of its
// largest group, relative to the share's own (half the mean size of the first tile, whatever single tokens hold).  A row's
// reference is the largest such product (as logit + size) in its first tile, or where it was last raised, and a weight is
// carried as 2^CK_LIFT times itself relative to it, so that a token with a large logit and small values (a sink) does not
// push the weights of those that make up the output out of fp16.  Where a size lies outside [CK_SIZE_LEAST, CK_SIZE_MOST]
// the weight also takes what it lies outside by (its level), and the values leave it.  So the largest product's weight
// stands at 2^0 to 2^12, 16 to 4 powers of two below fp16's end (at 2^2 for values of the mean size); bits are lost of
// products 2^-13 of it and less, and those below 2^-24 are gone.  (Without sizes, a sink of no values 20 nats above the
// others left the output 20 % off; with them 2K tokens of 32K take 938 us instead of 915, a 4K prompt 252 instead of 241.)
// Raising drains the stream's products: for a lift of 6, a 4K prompt takes 3 % longer.
constexpr float CK_LIFT = 3.f;
constexpr int CK_SIZE_LEAST = -9, CK_SIZE_MOST = 3, CK_SIZE_NONE = -90;  // (of zeros: sums of their weights stay below 2^93 a token)
constexpr int CK_SHARE_LEAST = -6, CK_SHARE_MOST = 11;  // (what values are brought to has its bits in fp16)
__device__ __forceinline__ int ck_size(float z, int share) { return max(CK_SIZE_NONE, (int)(__float_as_uint(z) >> 23) - 127 - share); }
__device__ __forceinline__ int ck_level(int size) { return size - max(CK_SIZE_LEAST, min(CK_SIZE_MOST, size)); }
// The same as fp32 numbers, without a conversion (2^23 + n by its bits).
__device__ __forceinline__ float ck_size_f(float z, float share_bias) { return fmaxf((float)CK_SIZE_NONE, __uint_as_float(0x4b000000u | __float_as_uint(z) >> 23) - share_bias); }
__device__ __forceinline__ float ck_level_f(float size) { return size - fmaxf((float)CK_SIZE_LEAST, fminf((float)CK_SIZE_MOST, size)); }
__device__ __forceinline__ float ck_pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
constexpr long long CK_SHORT_WAIT_CYCLES = 2000000LL;

// Rows [r0, r0 + rows) of sequence b (row = token * G + head of the group), and the pages
// that one of them sees: page x of the list is page x of the sequence below `sinks`, and
// page x + skip from there on.
struct __align__(16) CkBlock {
    int64_t start;   // of the blocks before it, per KV head: their cost
    int cost, tiles;
    int b, q0, n, ctx;
    int r0, rows, pages, sinks;
    int skip, index_in_b, pad0, pad1;
};
struct CkPlan {
    int blocks, ctas;
    int64_t total;  // cost of all heads
};

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
    CkPlan* plan;
    int64_t* cut;         // [ctas + 1]: where the cost of all heads is cut into shares
    CkBlock* block;       // [max_blocks]
    int max_blocks, block_rows;
    __half* rot;          // q' [H_kv][n_tok * G][D], channels in the order of the unpacked keys
    float* row_scale;     // [H_kv][n_tok * G]: logit = product * row_scale
    float* main;          // [H_kv * n_tok * G][PART_STRIDE] partials of the shares that begin a block
    float* second;        // of their second stream (blocks of one row tile)
    int64_t second_rows;  // rows of `second` per sequence and KV head (0: as in main)
    float* extra;         // [ctas][CK_ROWS][PART_STRIDE] of the shares that begin within one
    int ctas;
    int drop;
};

// ------------------------------------------------------------------ plan

// New tokens of sequence b: first row and count (0 where q_start is not what it should be).
__device__ __forceinline__ int2 ck_tokens(const ChunkArgs& a, int b) {
    const int s = __ldg(a.q_start + b), e = __ldg(a.q_start + b + 1);
    if (s < 0 || e < s || e > a.n_tok) {
        atomicOr(a.error, ERR_BAD_ROWS);
        return make_int2(0, 0);
    }
    return make_int2(s, e - s);
}
__device__ __forceinline__ int ck_blocks(const ChunkArgs& a, int n) { return (int)(((int64_t)n * a.G + a.block_rows - 1) / a.block_rows); }

__device__ __forceinline__ int ck_weight(int rows) { return rows > CK_ROW_TILE ? 2 : 1; }

__device__ __forceinline__ int64_t ck_scan(int64_t own, int64_t* warp_sums, int64_t& total) {  // exclusive, over the CTA's 256 threads
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    return before + inc - own;
}

// One CTA of 256 threads: a thread takes a run of sequences, then a block at a time.
__device__ void ck_make_plan(const ChunkArgs& a) {
    __shared__ int64_t sums[8];
    const int tid = threadIdx.x, per = (a.B + 255) / 256, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    // (in 64 bits: where the row starts go up and down, the sequences' blocks are more than max_blocks, even than 2^31)
    int64_t own = 0, all;
    for (int b = b0; b < b1; ++b) own += ck_blocks(a, ck_tokens(a, b).y);
    int64_t at = ck_scan(own, sums, all);
    for (int b = b0; b < b1; ++b) {
        const int2 t = ck_tokens(a, b);
        const int ctx = (int)min((int64_t)max(0, __ldg(a.context_lens + b)), (int64_t)a.max_pages * PAGE);
        for (int x = 0, n = ck_blocks(a, t.y); x < n && at < a.max_blocks; ++x, ++at) {
            CkBlock& k = a.block[at];
            k.b = b;
            k.q0 = t.x;
            k.n = t.y;
            k.ctx = ctx;
            k.index_in_b = x;
        }
    }
    __syncthreads();
    const int n_blocks = (int)min(all, (int64_t)a.max_blocks);
    int64_t base = 0;
    for (int e0 = 0; e0 < n_blocks; e0 += 256) {
        const int e = e0 + tid;
        CkBlock k = {};
        if (e < n_blocks) {
            k = a.block[e];
            k.r0 = k.index_in_b * a.block_rows;
            k.rows = (int)min((int64_t)a.block_rows, (int64_t)k.n * a.G - k.r0);
            const int first = k.ctx - k.n + k.r0 / a.G, last = k.ctx - k.n + (k.r0 + k.rows - 1) / a.G;  // positions
            k.pages = k.sinks = k.skip = k.tiles = k.cost = 0;
            if (last >= 0) {
                const int low = a.window ? max(0, first - min(first, a.window - 1)) : 0;  // (first < 0: from 0 on)
                const int fp = (first < 0 ? 0 : low) / PAGE;
                k.sinks = min(fp, (min(a.sinks, last + 1) + PAGE - 1) / PAGE);
                k.skip = fp - k.sinks;
                k.pages = last / PAGE + 1 - k.skip;
                k.tiles = (k.pages + CK_PAGES - 1) / CK_PAGES;
                k.cost = ck_weight(k.rows) * k.tiles + (a.block_rows == CK_ROWS ? CK_UNIT_COST : CK_UNIT_COST_FEW);
            }
        }
        int64_t total;
        k.start = base + ck_scan((int64_t)k.cost, sums, total);
        if (e < n_blocks) a.block[e] = k;
        base += total;
    }
    const int64_t least = a.block_rows == CK_ROWS ? CK_LEAST_SHARE : CK_LEAST_SHARE_FEW;
    const int64_t total = base * a.H_kv, C = min((int64_t)a.ctas, (total + least - 1) / least);
    for (int c = tid; c <= C; c += 256) a.cut[c] = C ? c * total / C : 0;
    if (tid == 0) {
        a.plan->blocks = n_blocks;
        a.plan->total = total;
        a.plan->ctas = (int)C;
    }
}

// A share: tiles [from, to) of head h of a block, out of cost [pos, end).
struct CkWalk {
    int64_t pos, end;
    int e, h, from, to;
    CkBlock k;
    __device__ __forceinline__ void read(const ChunkArgs& a) {
        const int4* p = reinterpret_cast<const int4*>(a.block + e);
        int4* q = reinterpret_cast<int4*>(&k);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __ldcg(p + i);
    }
    // The next share with tiles; false at the end.  (e, h) name the unit that holds pos.
    __device__ __forceinline__ bool next(const ChunkArgs& a) {
        while (pos < end) {
            read(a);
            if (k.cost == 0) {
                ++e;
                continue;
            }
            const int64_t unit = k.start * a.H_kv + (int64_t)h * k.cost;
            const int x0 = (int)(pos - unit), x1 = (int)min(end - unit, (int64_t)k.cost), w = ck_weight(k.rows);
            from = (x0 + w - 1) / w;
            to = min(k.tiles, (x1 + w - 1) / w);
            pos = unit + x1;
            last_h = h;
            if (x1 == k.cost && ++h == a.H_kv) {
                h = 0;
                ++e;
            }
            if (from < to) return true;
        }
        return false;
    }
    int last_h;  // head of the share that next() found
};

// ------------------------------------------------------------------ 1: rotate

// The rotations take one fp16 product each: a rotation's entries, the queries (8 bits of their own) and the outputs, each
// row brought to a power of two by its largest value, keep 11 bits, as do the rotated queries in any case, and an output
// is rounded to 8.  (With both factors in parts, three products, a prompt of 4K tokens and 32 heads took 57 us to finish.)
__device__ __forceinline__ uint32_t ck_pack(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
}
// Power of two that brings x into [2^to, 2^(to + 1)) (1 for 0 and what is not finite), of any size: itself at least 2^-127.
__device__ __forceinline__ float ck_scale(float x, int to) { return x > 0.f && x < CUDART_INF_F ? ldexpf(1.f, min(126, to - ilogbf(x))) : 1.f; }

// A matrix as the B operand of m16n8k16: [K step][8 columns][lane].  What a product sums over may come in any order: that of
// the K steps is such that lane t of a row's four loads its values of a step (or of two) at once.
struct __align__(16) CkMatrix {
    uint2 f[8][16][32];
};

// Position of a key channel in the unpacked keys: a word's eight channels come as (0, 4), (1, 5), (2, 6), (3, 7).
__host__ __device__ constexpr int ck_key_at(int ch) { return (ch & ~7) | (ch & 3) << 1 | (ch >> 2 & 1); }
// (A value channel 32 g + 4 r + i stands at 32 g + 8 i + r.)

// CTAs of 256 threads, 128 rows each (a warp 16); the last CTA of a head's row makes the plan.  4096 tokens of 32 heads:
// 33 us for 67 MB (10 at the copy rate), the matrix's way into the operands' layout and a tile or two behind it.
struct __align__(16) CkRotate {
    CkMatrix R;
    __align__(16) __half out[8][16][D / 2 + 8];  // half a row at a time, so that four CTAs share an SM
};
__global__ void __launch_bounds__(256, 4) chunk_rotate_kernel(const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    CkRotate& sm = *reinterpret_cast<CkRotate*>(smem_raw);
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0) ck_make_plan(a);
        return;
    }
    const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const float* Rk = a.Rk + (size_t)h * D * D;
    const int64_t rows = (int64_t)a.n_tok * a.G;
    const float unit = a.scale_log2 < 0.f ? -1.f : a.scale_log2 > 0.f ? 1.f : a.scale_log2;  // (NaN stays NaN)
    auto fetch = [&](int64_t r0, uint32_t (&x)[8][4]) {
        const __nv_bfloat16* q[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t row = min(r0 + r + 8 * e, rows - 1);
            q[e] = a.q + ((row / a.G) * a.H_q + (int64_t)h * a.G + row % a.G) * D;
        }
#pragma unroll
        for (int ks = 0; ks < 8; ks += 2)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // channels 8 t .. 8 t + 7 of 32: four of a K step, then four of the next
                const uint4 y = __ldg(reinterpret_cast<const uint4*>(q[e] + 16 * ks + 8 * t));
                x[ks][e] = y.x;
                x[ks][e + 2] = y.y;
                x[ks + 1][e] = y.z;
                x[ks + 1][e + 2] = y.w;
            }
    };
    uint32_t x[8][4];
    int64_t r0 = (int64_t)blockIdx.x * 128 + 16 * warp;
    if (r0 < rows) fetch(r0, x);
    // Columns of the product in the order of the unpacked keys: position n holds channel c with ck_key_at(c) == n.
    // A thread takes four channels (low or high half of eight: positions 2 i or 2 i + 1) of four rows.  (A lane's place is
    // turned by the column set, so that a warp's stores meet all banks.)
#pragma unroll 2
    for (int y = threadIdx.x; y < 8 * 4 * 32; y += 256) {
        const int c4 = (y & 7) | (y >> 2 & 0x18), tt = (y >> 3) & 3, ks = y >> 7;
        const float* p = Rk + (size_t)(32 * (ks >> 1) + 8 * tt + 4 * (ks & 1)) * D + 4 * c4;
        float k[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p + j * D));
            k[j][0] = v.x, k[j][1] = v.y, k[j][2] = v.z, k[j][3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sm.R.f[ks][c4 >> 1][(4 * (2 * i + (c4 & 1)) + tt) ^ 8 * (c4 >> 1 & 3)] = make_uint2(pack_half2(k[0][i], k[1][i]), pack_half2(k[2][i], k[3][i]));
    }
    __syncthreads();
    for (; r0 < rows; r0 += (int64_t)(gridDim.x - 1) * 128) {
        // a row's largest value to 1..2: its rotated ones stay within 2^4.5 times R_k's norm, in fp16 for one of up to 2^11, and
        // lose nothing that counts at fp16's other end, 2^-25, for one down to 2^-11 (the sign of the logits' scale goes into
        // the queries, so that row_scale is positive)
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x[ks][e])));
                m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x[ks][e + 2])));
            }
            float top = fmaxf(__low2float(m), __high2float(m));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float sigma = ck_scale(top, 0);
            f[e] = unit * sigma;
            const int64_t row = r0 + r + 8 * e;
            if (t == 0 && row < rows) a.row_scale[(int64_t)h * rows + row] = unit == 0.f ? 1.f : fmaxf(fabsf(a.scale_log2) / sigma, 1e-30f);
        }
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[ks][e] = pack_half2(__uint_as_float(x[ks][e] << 16) * f[e & 1], __uint_as_float(x[ks][e] & 0xffff0000u) * f[e & 1]);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
#pragma unroll 4
            for (int nt = 0; nt < 8; ++nt) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint2 b = sm.R.f[ks][8 * part + nt][lane ^ 8 * (nt & 3)];
                    mma_f16_16816(c, x[ks], b.x, b.y);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) *reinterpret_cast<uint32_t*>(&sm.out[warp][r + 8 * e][8 * nt + 2 * t]) = pack_half2(c[2 * e], c[2 * e + 1]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // four rows at a time, 16 bytes a lane
                const int y = 4 * i + (lane >> 3);
                if (r0 + y < rows)
                    *reinterpret_cast<uint4*>(a.rot + ((int64_t)h * rows + r0 + y) * D + 64 * part + 8 * (lane & 7)) = lds128(&sm.out[warp][y][8 * (lane & 7)]);
            }
            __syncwarp();
        }
        const int64_t next = r0 + (int64_t)(gridDim.x - 1) * 128;
        if (next < rows) fetch(next, x);
    }
}

// ------------------------------------------------------------------ 2: stream
//
// Two warpgroups of softmax (a thread a row of its row tile), four that unpack, two warps that
// issue products and one that fetches pages.  A block of more than 128 rows has two row
// tiles, whose warpgroups both take every tile of tokens; a block of up to 128 has one, and
// the warpgroups take every other tile of tokens of it (two streams, each with sums of its
// own).  In either case the products of one stream run while the other one's softmax does.
//
// 2048 tokens of 32K, 32 q / 8 KV heads: 0.94 ms, 1.14 PFLOP/s, 0.57 of a library product's rate.  Bound by the roles'
// instructions and their waits together: tensor pipe 44 %, issue 56 %; alone, of 1010 us, the products took 783, the
// softmax 802 and the unpacking 620.  (With 128 logit columns a product and one buffer a stream, for which tensor memory
// has room, products alone took 637 us, and all of it 1164.)
//
//   TMEM     S [stream][2 buffers] (the logits of a tile, and over them its weights P as
//            fp16), O [stream]
//   shared   Q [stream], K [4 stages] and V [2] as K-major operands in the 128-byte swizzle
//            (V transposed: rows are channels), six raw stages; FEW: one Q, four stages of V
constexpr int CK_QUERIES = CK_ROW_TILE * D * 2, CK_OPERAND = CK_TILE * D * 2;  // bytes
constexpr int CK_RAW = CK_PAGES * INT4_TILE, CK_INFOS = 8, CK_SHARES = 4;
constexpr int CK_SOFTMAX = 8, CK_UNPACK = 16;  // warps
// (Registers: 896 threads of 72 at launch; 128 for softmax, 48 for unpacking and 56 for the rest are those 64512.)
constexpr int CK_THREADS = 32 * (CK_SOFTMAX + CK_UNPACK + 4);

struct __align__(16) CkInfo {  // of a tile of tokens, written with its keys
    int base[4];          // first position of each page, -1 without one
    uint32_t marks[4];    // tokens of each page: bits 0..15 values that are not finite, bits 16..31 keys carried at 2^-4
    uint32_t flags[4];    // of each page: 1 there are marks, 2 there are levels
    float z[CK_TILE];     // 8 |scale| + |min| of each token's values
    uint32_t special;     // bit t: stream t's rows do not all see all of it
    float share_bias;     // the share's size + 127 + 2^23
};
struct __align__(16) CkShare {  // what the roles need of a share
    int n, two, from, rows;     // tiles; two row tiles; from > 0: not the block's first share
    int again;                  // a further run of the same share
    int r0, pos0, ctx, b;       // pos0: position of the sequence's first new token
    int first[2], last[2];      // positions of the streams' first and last rows
    int64_t row0;               // the sequence's first row among all of a head's
    int h, end;
};
// FEW: blocks of one row tile only.  One copy of the queries serves both streams, and more raw stages cover the
// cache's latency, which bounds such calls (8 x 5 tokens at 32K: 208 us with three raw stages, 196 with six).
template <bool FEW>
struct __align__(1024) CkSmem {
    static constexpr int K_STAGES = 4, V_STAGES = FEW ? 4 : 2, RAW_STAGES = 6;
    // (A tile's stages are its number modulo their count.  The warps of the even tiles never wait for an odd one's phase:
    // with an odd count they could ask for a stage's next phase while the last one is open, and be let through.)
    // (A tile's keys come with what the softmax reads of it, in the place of the tile CK_INFOS before.  They wait for the
    // logits of the tile K_STAGES before, which their stream forms after the softmax of its second tile before that one:
    // 2 K_STAGES before, where streams take every other tile, K_STAGES + 2 where they take all.)
    static_assert(CK_INFOS >= 2 * K_STAGES && CK_INFOS >= K_STAGES + 2, "the softmax is done with an info's place");
    static_assert(RAW_STAGES % 2 == 0 && K_STAGES % 2 == 0 && V_STAGES % 2 == 0, "even and odd tiles have stages of their own");
    uint8_t q[FEW ? 1 : 2][CK_QUERIES], k[K_STAGES][CK_OPERAND], v[V_STAGES][CK_OPERAND];
    uint8_t raw[RAW_STAGES][CK_RAW];
    CkInfo info[CK_INFOS];
    CkShare share[CK_SHARES];
    int share_size[CK_SHARES];  // (known with the share's first tile)
    float2 share_band[CK_SHARES];  // the sizes z without a level: from .x on, below .y
    __align__(16) int raw_base[RAW_STAGES][CK_PAGES];
    uint64_t raw_full[RAW_STAGES], raw_free[RAW_STAGES], k_full[K_STAGES], k_free[K_STAGES], v_full[V_STAGES], v_free[V_STAGES];
    uint64_t q_full[CK_SHARES], q_free, s_full[2][2], p_full[2][2], o_done[2][2], o_full[2], drained[2], share_full[CK_SHARES], share_free[CK_SHARES];
    uint32_t tmem;
    int dead;
    uint32_t stages;  // raw stages fetched
};
static_assert(sizeof(CkSmem<false>) + 1024 <= 227 * 1024 && sizeof(CkSmem<true>) + 1024 <= 227 * 1024, "chunk shared memory above 227 KB");

// Descriptor of an operand, K-major in the 128-byte swizzle: atoms of 8 rows, 1024 bytes apart.  Its low word holds the
// address in 16-byte units.
__device__ __forceinline__ uint32_t ck_desc_lo(const void* p) { return (smem_u32(p) & 0x3ffff) >> 4 | 1u << 16; }
constexpr uint32_t CK_DESC_HI = (1024 >> 4) | 1u << 14 | 2u << 29;

__device__ __forceinline__ bool ck_elect() {
    uint32_t x;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
    return x != 0;
}
// fp32 accumulators, fp16 operands, both K-major, 128 rows, 128 columns or 64
constexpr uint32_t CK_IDESC = 1u << 4 | (128u >> 3) << 17 | (128u >> 4) << 24, CK_IDESC_QK = 1u << 4 | (64u >> 3) << 17 | (128u >> 4) << 24;

__device__ __forceinline__ void ck_mma_ss(uint32_t d, uint32_t a, uint32_t b, bool add, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add),
        "r"(CK_DESC_HI)
        : "memory");
}
__device__ __forceinline__ void ck_mma_ts(uint32_t d, uint32_t a, uint32_t b, bool add, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n mov.b64 y, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add),
        "r"(CK_DESC_HI)
        : "memory");
}
__device__ __forceinline__ void ck_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void ck_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void ck_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// What was loaded is used after the wait only (it passes through it).
#define CK_T8(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]), "+r"(x[i + 4]), "+r"(x[i + 5]), "+r"(x[i + 6]), "+r"(x[i + 7])
__device__ __forceinline__ void ck_loaded16(uint32_t* x) { asm volatile("tcgen05.wait::ld.sync.aligned;" : CK_T8(x, 0), CK_T8(x, 8)::"memory"); }
__device__ __forceinline__ void ck_loaded32(uint32_t* x) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : CK_T8(x, 0), CK_T8(x, 8), CK_T8(x, 16), CK_T8(x, 24)::"memory");
}
__device__ __forceinline__ void ck_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define CK_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define CK_W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
__device__ __forceinline__ void ck_tmem_ld32(uint32_t* x, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : CK_R8(x, 0), CK_R8(x, 8), CK_R8(x, 16), CK_R8(x, 24)
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void ck_tmem_ld16(uint32_t* x, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : CK_R8(x, 0), CK_R8(x, 8)
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void ck_tmem_st32(const uint32_t* x, uint32_t at) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::CK_W8(x, 0),
        CK_W8(x, 8), CK_W8(x, 16), CK_W8(x, 24), "r"(at)
        : "memory");
}
__device__ __forceinline__ void ck_tmem_st16(const uint32_t* x, uint32_t at) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::CK_W8(x, 0),
        CK_W8(x, 8), "r"(at)
        : "memory");
}
__device__ __forceinline__ float ck_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ck_fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n fma.rn.f32x2 x, x, y, z;\n"
        " mov.b64 {%0, %1}, x;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 ck_add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Codes of a word as fp16 numbers, two at a time: nibbles (0, 4), (1, 5), (2, 6), (3, 7).  1024 + c by its bits, less 1024.
// (The constants stand in registers that the compiler does not see through: otherwise it takes two instructions for an AND
// and an OR with two immediates, and moves the others again for each word.)
struct CkConst {
    uint32_t low, high, magic, one, sixteenth, back;
    __device__ __forceinline__ CkConst() {
        asm volatile("mov.b32 %0, 0x000f000f;\n mov.b32 %1, 0x00f000f0;\n mov.b32 %2, 0x64006400;\n mov.b32 %3, 0xe400e400;\n mov.b32 %4, 0x2c002c00;\n mov.b32 %5, 0xd400d400;"
                     : "=r"(low), "=r"(high), "=r"(magic), "=r"(one), "=r"(sixteenth), "=r"(back));  // .. 1024, -1024, 1/16, -64
    }
    __device__ __forceinline__ __half2 take(uint32_t w, uint32_t mask) const {
        uint32_t x;
        asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w), "r"(mask), "r"(magic));
        return u32_as_h2(x);
    }
    __device__ __forceinline__ void codes(uint32_t w, __half2 (&c)[4]) const {
        const uint32_t v = w >> 8;
        c[0] = __hadd2(take(w, low), u32_as_h2(one));
        c[1] = __hfma2(take(w, high), u32_as_h2(sixteenth), u32_as_h2(back));
        c[2] = __hadd2(take(v, low), u32_as_h2(one));
        c[3] = __hfma2(take(v, high), u32_as_h2(sixteenth), u32_as_h2(back));
    }
};

// Largest of four groups' scales or mins of a slot pair; NaN where one is.
__device__ __forceinline__ __half2 ck_most(uint4 y) {
    return __hmax2_nan(__hmax2_nan(__habs2(u32_as_h2(y.x)), __habs2(u32_as_h2(y.y))), __hmax2_nan(__habs2(u32_as_h2(y.z)), __habs2(u32_as_h2(y.w))));
}
__device__ __forceinline__ float2 ck_sizes(__half2 scale, __half2 min) {
    const float2 s = __half22float2(scale), m = __half22float2(min);
    return make_float2(fmaf(8.f, s.x, m.x), fmaf(8.f, s.y, m.y));
}
// Whether the keys of a token's scales and mins might leave fp16.
__device__ __forceinline__ bool ck_big_keys(uint4 meta) {
    const __half2 s = __hmax2_nan(__habs2(u32_as_h2(meta.x)), __habs2(u32_as_h2(meta.y)));
    const __half2 m = __hmax2_nan(__habs2(u32_as_h2(meta.z)), __habs2(u32_as_h2(meta.w)));
    return !(__hblt2(s, __float2half2_rn(2048.f)) && __hblt2(m, __float2half2_rn(32768.f)));
}

template <bool FEW>
__global__ void __launch_bounds__(CK_THREADS, 1) chunk_stream_kernel(const __grid_constant__ ChunkArgs a) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int CK_RAW_STAGES = CkSmem<FEW>::RAW_STAGES, CK_K_STAGES = CkSmem<FEW>::K_STAGES, CK_V_STAGES = CkSmem<FEW>::V_STAGES;
    CkSmem<FEW>& sm = *reinterpret_cast<CkSmem<FEW>*>(smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < CK_RAW_STAGES; ++i) {
            mbar_init(&sm.raw_full[i], 1);
            mbar_init(&sm.raw_free[i], CK_UNPACK / 2);
        }
        for (int i = 0; i < CK_K_STAGES; ++i) {
            mbar_init(&sm.k_full[i], CK_UNPACK / 4);
            mbar_init(&sm.k_free[i], 2);
        }
        for (int i = 0; i < CK_V_STAGES; ++i) {
            mbar_init(&sm.v_full[i], CK_UNPACK / 4);
            mbar_init(&sm.v_free[i], 2);
        }
        mbar_init(&sm.q_free, CK_SOFTMAX);
        for (int i = 0; i < 2; ++i) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sm.s_full[i][h], 1);
                mbar_init(&sm.p_full[i][h], 4);
                mbar_init(&sm.o_done[i][h], 1);
            }
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.drained[i], 1);
        }
        for (int i = 0; i < CK_SHARES; ++i) {
            mbar_init(&sm.share_full[i], 1);
            mbar_init(&sm.q_full[i], CK_SOFTMAX);
            mbar_init(&sm.share_free[i], CK_SOFTMAX + CK_UNPACK + 2);  // the warps but the loader
        }
        sm.dead = 0;
        sm.stages = 0;
        fence_mbar_init();
    }
    if (warp == CK_SOFTMAX + CK_UNPACK) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    ck_fence_before();
    __syncthreads();
    ck_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = sm.tmem;
    const long long limit = a.drop ? CK_SHORT_WAIT_CYCLES : WAIT_LIMIT_CYCLES;
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // a whole warp
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        bool ok = true;
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, parity)) {
            if (*(volatile int*)&sm.dead) {
                ok = false;
                break;
            }
            if (clock64() - t0 > limit) {
                *(volatile int*)&sm.dead = 1;
                atomicOr(a.error, ERR_TIMEOUT);
                ok = false;
                break;
            }
        }
        return (bool)__all_sync(0xffffffffu, ok);
    };
    // the shares, as the loader finds them; false at the end
    uint32_t n_share = 0;
    auto next_share = [&]() {
        if (n_share) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.share_free[(n_share - 1) % CK_SHARES]);
        }
        const bool ok = wait(&sm.share_full[n_share % CK_SHARES], (n_share / CK_SHARES) & 1) && !sm.share[n_share % CK_SHARES].end;
        ++n_share;
        return ok;
    };

    if (warp >= CK_SOFTMAX + CK_UNPACK) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (!(warp & 1)) {
            // ---- products of stream t.  Its logits stand in two buffers: the next tile's are formed while the softmax works
            // on this one's.  (Two warps: the tensor core takes few products in advance, so one warp's waits between two
            // streams' products left it idle.)  The whole warp goes along, so that descriptors stay in uniform registers;
            // one lane issues.
            const int t = __shfl_sync(0xffffffffu, warp >> 1 & 1, 0);
            uint32_t tile0 = 0, done = 0;  // tiles before this share, of this stream
            bool ok = true;
            const bool leader = ck_elect();
            const uint32_t q_lo = ck_desc_lo(sm.q[FEW ? 0 : t]), k_lo = ck_desc_lo(sm.k[0]), v_lo = ck_desc_lo(sm.v[0]);
            const uint32_t s_at = tmem + 128 * t, o_at = tmem + 256 + 128 * t;
            while (ok && next_share()) {
                const CkShare& g = sm.share[(n_share - 1) % CK_SHARES];
                const int n = __shfl_sync(0xffffffffu, g.n, 0), two = __shfl_sync(0xffffffffu, g.two, 0), ns = two ? n : (n + 1 - t) / 2;
                // both streams' queries: then both are done with the shares before, and every phase of a stage that this
                // stream's tiles have not been in is over
                ok = wait(&sm.q_full[(n_share - 1) % CK_SHARES], (n_share - 1) / CK_SHARES & 1);
#pragma unroll 1
                for (int x = 0; x < ns + 2 && ok; ++x) {
                    if (x >= 2) {  // the weighted sum of tile x - 2
                        const uint32_t tile = tile0 + (two ? x - 2 : 2 * (x - 2) + t), st = tile % CK_V_STAGES, step = done + x - 2;
                        if (!(ok = wait(&sm.v_full[st], tile / CK_V_STAGES & 1) && wait(&sm.p_full[t][step & 1], step >> 1 & 1))) break;
                        ck_fence_after();
                        if (leader) {
                            const uint32_t vd = v_lo + st * (CK_OPERAND >> 4), p_at = s_at + 64 * (step & 1);
                            ck_mma_ts(o_at, p_at, vd, x > 2, CK_IDESC);
#pragma unroll
                            for (int i = 1; i < 4; ++i) ck_mma_ts(o_at, p_at + 8 * i, vd + 2 * i, true, CK_IDESC);
                            ck_commit(&sm.o_done[t][step & 1]);
                            if (x == ns + 1) ck_commit(&sm.o_full[t]);
                            ck_commit(&sm.v_free[st]);
                            if (!two) ck_commit(&sm.v_free[st]);
                        }
                        __syncwarp();
                    }
                    if (x < ns) {  // the logits of tile x
                        const uint32_t tile = tile0 + (two ? x : 2 * x + t), st = tile % CK_K_STAGES, step = done + x;
                        if (!(ok = wait(&sm.k_full[st], tile / CK_K_STAGES & 1))) break;
                        ck_fence_after();
                        if (leader) {
                            const uint32_t kd = k_lo + st * (CK_OPERAND >> 4);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                ck_mma_ss(s_at + 64 * (step & 1), q_lo + (i & 3) * 2 + (i >> 2) * (CK_QUERIES >> 5), kd + (i & 3) * 2 + (i >> 2) * (CK_OPERAND >> 5),
                                          i > 0, CK_IDESC_QK);
                            ck_commit(&sm.s_full[t][step & 1]);
                            ck_commit(&sm.k_free[st]);
                            if (!two) ck_commit(&sm.k_free[st]);
                        }
                        __syncwarp();
                    }
                }
                tile0 += n;
                done += ns;
            }
            // everything issued is done before TMEM is freed
            if (leader) {
                ck_commit(&sm.drained[t]);
                (void)mbar_wait_bounded(&sm.drained[t], 0, 100000000LL);
            }
        } else if (warp == CK_SOFTMAX + CK_UNPACK + 1) {
            // ---- shares and pages
            const int C = __ldcg(&a.plan->ctas), cta = blockIdx.x, n_blocks = __ldcg(&a.plan->blocks);
            CkWalk w;
            w.pos = w.end = 0;
            w.e = w.h = 0;
            if (cta < C) {  // the block that holds pos: 33 cuts of the range at a time
                w.pos = __ldcg(a.cut + cta);
                w.end = __ldcg(a.cut + cta + 1);
                int lo = 0, hi = n_blocks;  // start[lo] * H <= pos, start[hi] * H > pos
                while (hi - lo > 1) {
                    const int step = (hi - lo + 32) / 33, x = lo + (lane + 1) * step;
                    const bool below = x < hi && __ldcg(&a.block[x].start) * a.H_kv <= w.pos;
                    const int n = __popc(__ballot_sync(0xffffffffu, below));
                    hi = min(hi, lo + (n + 1) * step);
                    lo += n * step;
                }
                // (of blocks with one start only the last costs anything, and the search ends there)
                w.e = lo;
                w.h = (int)((w.pos - __ldcg(&a.block[lo].start) * a.H_kv) / max(1, __ldcg(&a.block[lo].cost)));
            }
            uint32_t stage = 0;
            bool ok = true;
            const bool leader = ck_elect();
            int run = 0, to = 0;  // tiles of the share that are still to come
            for (uint32_t x = 0; ok; ++x) {
                bool have = run < to;
                if (!have && (have = w.next(a))) {
                    run = w.from;
                    to = w.to;
                }
                const int n = min(to - run, CK_RUN);
                if (x >= CK_SHARES && !(ok = wait(&sm.share_free[x % CK_SHARES], (x / CK_SHARES - 1) & 1))) break;
                if (lane == 0) {
                    CkShare& g = sm.share[x % CK_SHARES];
                    g.end = !have;
                    if (have) {
                        g.n = n;
                        g.again = run > w.from;
                        g.two = w.k.rows > CK_ROW_TILE;
                        g.from = w.from;
                        g.rows = w.k.rows;
                        g.r0 = w.k.r0;
                        g.pos0 = w.k.ctx - w.k.n;
                        g.ctx = w.k.ctx;
                        g.b = w.k.b;
                        g.h = w.last_h;
                        g.row0 = (int64_t)w.k.q0 * a.G;
                        for (int t = 0; t < 2; ++t) {
                            const int r0 = w.k.r0 + (g.two ? CK_ROW_TILE * t : 0), r1 = min(w.k.r0 + w.k.rows, r0 + CK_ROW_TILE) - 1;
                            g.first[t] = g.pos0 + r0 / a.G;
                            g.last[t] = g.pos0 + r1 / a.G;
                        }
                    }
                    mbar_arrive(&sm.share_full[x % CK_SHARES]);
                }
                __syncwarp();
                if (!have) break;
                // a lane's page of the next eight tiles' 32: its first position (-1: none, or a bad entry) and where it stands
                const int p0 = CK_PAGES * run, p1 = min(w.k.pages, CK_PAGES * (run + n)), sinks = w.k.sinks, skip = w.k.skip;
                run += n;
                const int32_t* table = a.block_table + (size_t)w.k.b * a.max_pages;
                auto ids = [&](int first) {
                    const int p = first + lane;
                    return p < p1 ? __ldg(table + p + (p < sinks ? 0 : skip)) : 0;
                };
                int next_id = ids(p0), base = -1;
                uint64_t from = 0;
                for (int s = 0; s < n; ++s, ++stage) {
                    if ((s & 7) == 0) {
                        const int p = p0 + CK_PAGES * s + lane;
                        const bool good = p < p1 && next_id >= 0 && (int64_t)next_id < a.num_pages;
                        if (p < p1 && !good) atomicOr(a.error, ERR_BAD_PAGE);
                        base = good ? PAGE * (p + (p < sinks ? 0 : skip)) : -1;
                        from = reinterpret_cast<uint64_t>(a.cache + ((size_t)(good ? next_id : 0) * a.H_kv + w.last_h) * INT4_TILE);
                        next_id = ids(p0 + CK_PAGES * s + 32);
                    }
                    const uint32_t slot = stage % CK_RAW_STAGES;
                    int at[CK_PAGES];
                    uint64_t src[CK_PAGES];
                    uint32_t bytes = 0;
#pragma unroll
                    for (int i = 0; i < CK_PAGES; ++i) {
                        at[i] = __shfl_sync(0xffffffffu, base, 4 * (s & 7) + i);
                        src[i] = __shfl_sync(0xffffffffu, from, 4 * (s & 7) + i);
                        bytes += at[i] >= 0 ? INT4_TILE : 0;
                    }
                    if (stage >= CK_RAW_STAGES && !(ok = wait(&sm.raw_free[slot], (stage / CK_RAW_STAGES - 1) & 1))) break;
                    if (leader) {
                        *reinterpret_cast<int4*>(sm.raw_base[slot]) = make_int4(at[0], at[1], at[2], at[3]);
#pragma unroll
                        for (int i = 0; i < CK_PAGES; ++i)
                            if (at[i] >= 0 && !(a.drop && stage == 0 && i == 0 && cta == 0))
                                bulk_g2s(sm.raw[slot] + i * INT4_TILE, reinterpret_cast<const void*>(src[i]), INT4_TILE, &sm.raw_full[slot]);
                    }
                    __syncwarp();
                    if (s == 0) {  // the share's size, while the first tile is on its way: a lane looks at a slot pair of a page
                        const int first = __shfl_sync(0xffffffffu, base, lane >> 3);
                        const uint8_t* y = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, from, lane >> 3)) + O4_VS + 16 * (lane & 7);
                        const int left = first < 0 ? 0 : w.k.ctx - first - 2 * (lane & 7);  // tokens of the pair
                        int size = 0, count = 0;
                        if (left > 0) {
                            const float2 z = ck_sizes(ck_most(__ldg(reinterpret_cast<const uint4*>(y))), ck_most(__ldg(reinterpret_cast<const uint4*>(y + O4_VM - O4_VS))));
                            if (z.x > 0.f && z.x < CUDART_INF_F) size = ck_size(z.x, 0), count = 1;
                            if (left > 1 && z.y > 0.f && z.y < CUDART_INF_F) size += ck_size(z.y, 0), ++count;
                        }
                        size = __reduce_add_sync(0xffffffffu, size);
                        count = __reduce_add_sync(0xffffffffu, count);
                        size = count ? max(CK_SHARE_LEAST, min(CK_SHARE_MOST, __float2int_rn((float)size / (float)count) - 1)) : 0;
                        if (lane == 0) {
                            sm.share_size[x % CK_SHARES] = size;
                            sm.share_band[x % CK_SHARES] = make_float2(ck_pow2(CK_SIZE_LEAST + size), ck_pow2(CK_SIZE_MOST + 1 + size));
                        }
                        __syncwarp();
                    }
                    if (leader) mbar_arrive_expect_tx(&sm.raw_full[slot], bytes);
                    __syncwarp();
                }
            }
            if (lane == 0) sm.stages = stage;
        }
    } else if (warp >= CK_SOFTMAX) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        // (keys on two of the four schedulers and values on the others: with both, and the softmax, on each, warps waited
        // for instructions more than for anything else)
        // Four warps take the even tiles of tokens and four the odd ones: a warp's chain of waits, loads and stores over one
        // tile covers another's.
        const int part = (warp & 1) | (warp - CK_SOFTMAX) >> 2 & 2;
        const uint32_t odd = (warp - CK_SOFTMAX) >> 2 & 1;
        uint32_t tile = 0;
        bool ok = true;
        const CkConst cc;
        if (!(warp & 2)) {
            // ---- keys: a thread takes the words t of all groups of two tokens
            const int t = lane & 3, tok = 16 * part + ((lane >> 3) ^ (lane & 4 ? 5 : 0));
            const uint32_t from = part * INT4_TILE + O4_KC + 64 * (tok & 15) + 16 * t, meta_from = part * INT4_TILE + O4_KM + 16 * (tok & 15);
            const uint32_t to0 = tok * 128 + ((t ^ (tok & 7)) << 4), to1 = tok * 128 + (((4 + t) ^ (tok & 7)) << 4);
            while (ok && next_share()) {
                const CkShare& share = sm.share[(n_share - 1) % CK_SHARES];
                for (int i = share.n; i > 0; --i, ++tile) {
                    if ((tile & 1) != odd) continue;
                    const uint32_t st = tile % CK_K_STAGES, slot = tile % CK_RAW_STAGES;
                    if (!(ok = wait(&sm.raw_full[slot], tile / CK_RAW_STAGES & 1))) break;
                    if (tile >= CK_K_STAGES && !(ok = wait(&sm.k_free[st], (tile / CK_K_STAGES - 1) & 1))) break;
                    CkInfo& info = sm.info[tile % CK_INFOS];
                    bool big = false;  // some keys of the page might leave fp16
                    {   // a warp looks at a page first: a lane at a token's keys, and at a slot pair's scales or mins of the values
                        const uint8_t* page = sm.raw[slot] + part * INT4_TILE + 16 * (lane & 15);
                        const uint4 keys = lds128(page + O4_KM);
                        const __half2 most = ck_most(lds128(page + O4_VS)), they = u32_as_h2(__shfl_xor_sync(0xffffffffu, h2_as_u32(most), 8));
                        const float2 z = lane & 8 ? ck_sizes(they, most) : ck_sizes(most, they), band = sm.share_band[(n_share - 1) % CK_SHARES];
                        const int pair = 2 * (lane & 7);
                        if (lane < 8) *reinterpret_cast<float2*>(info.z + PAGE * part + pair) = z;
                        const bool usual = __hblt2(ck_most(keys), __float2half2_rn(2048.f)) && z.x >= band.x && z.x < band.y && z.y >= band.x && z.y < band.y;
                        uint32_t flags = 0;
                        if (!__all_sync(0xffffffffu, usual)) {  // huge keys, values that are not finite or of another size than most
                            const int left = sm.raw_base[slot][part] < 0 ? 0 : share.ctx - sm.raw_base[slot][part];
                            uint32_t marks = ck_big_keys(keys) ? 0x10000u << (lane & 15) : 0u;
                            big = __any_sync(0xffffffffu, marks);
                            marks |= ((z.x < CUDART_INF_F ? 0u : 1u) | (z.y < CUDART_INF_F ? 0u : 2u)) << pair;
                            marks = __reduce_or_sync(0xffffffffu, marks);
                            const bool out = (pair < left && !(z.x >= band.x && z.x < band.y)) || (pair + 1 < left && !(z.y >= band.x && z.y < band.y));
                            flags = (left > 0 && marks ? 1u : 0u) | (__any_sync(0xffffffffu, out) ? 2u : 0u);
                            if (lane == 0) info.marks[part] = marks;
                        }
                        if (lane == 0) info.flags[part] = flags;
                    }
#pragma unroll 1
                    for (int e = 0; e < 2; ++e) {  // tokens tok and tok + 8
                        const uint4 codes = lds128(sm.raw[slot] + from + 512 * e);
                        uint4 meta = lds128(sm.raw[slot] + meta_from + 128 * e);
                        const uint32_t word[4] = {codes.x, codes.y, codes.z, codes.w};
                        // min + code * scale is exact or has its 11 bits at any size.  A token whose scales reach 2^11 or whose mins
                        // reach 2^15 might leave fp16: its keys are carried at 2^-4, and its logits times 2^4 in the softmax.
                        if (big) {
                            const __half2 f = ck_big_keys(meta) ? u32_as_h2(cc.sixteenth) : __float2half2_rn(1.f);
                            meta.x = h2_as_u32(__hmul2(u32_as_h2(meta.x), f));
                            meta.y = h2_as_u32(__hmul2(u32_as_h2(meta.y), f));
                            meta.z = h2_as_u32(__hmul2(u32_as_h2(meta.z), f));
                            meta.w = h2_as_u32(__hmul2(u32_as_h2(meta.w), f));
                        }
                        const __half2 s01 = u32_as_h2(meta.x), s23 = u32_as_h2(meta.y), m01 = u32_as_h2(meta.z), m23 = u32_as_h2(meta.w);
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const __half2 s = g & 1 ? __high2half2(g < 2 ? s01 : s23) : __low2half2(g < 2 ? s01 : s23);
                            const __half2 m = g & 1 ? __high2half2(g < 2 ? m01 : m23) : __low2half2(g < 2 ? m01 : m23);
                            __half2 c[4];
                            cc.codes(word[g], c);
                            *reinterpret_cast<uint4*>(sm.k[st] + (g >> 1) * (CK_OPERAND / 2) + (g & 1 ? to1 : to0) + 1024 * e) =
                                make_uint4(h2_as_u32(__hfma2(c[0], s, m)), h2_as_u32(__hfma2(c[1], s, m)), h2_as_u32(__hfma2(c[2], s, m)),
                                           h2_as_u32(__hfma2(c[3], s, m)));
                        }
                    }
                    if (part == 0) {
                        const int at = sm.raw_base[slot][lane & 3];
                        bool cut[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            cut[x] = at < 0 || at + PAGE - 1 > share.first[x] || (a.window && at <= share.last[x] - a.window && at + PAGE > a.sinks);
                        const uint32_t s0 = __any_sync(0xffffffffu, cut[0]), s1 = __any_sync(0xffffffffu, cut[1]);
                        if (lane < 4) info.base[lane] = at;
                        if (lane == 0) {
                            info.special = s0 | s1 << 1;
                            info.share_bias = (float)(sm.share_size[(n_share - 1) % CK_SHARES] + 127 + (1 << 23));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.raw_free[slot]);
                        mbar_arrive(&sm.k_full[st]);
                    }
                }
            }
        } else {
            // ---- values: a thread takes the words r of eight tokens and two groups
            const int r = lane & 7, oct = 4 * (part & 1) + (lane >> 3), g0 = part & 2, pair0 = 4 * (oct & 1);
            const uint32_t from = (oct >> 1) * INT4_TILE + O4_VC + 128 * pair0 + 16 * r + 4 * g0, meta_from = (oct >> 1) * INT4_TILE + O4_VS + 16 * pair0 + 4 * g0;
            const uint32_t to = (32 * g0 + r) * 128 + ((oct ^ r) << 4);
            while (ok && next_share()) {
                const CkShare& share = sm.share[(n_share - 1) % CK_SHARES];
                for (int i = share.n; i > 0; --i, ++tile) {
                    if ((tile & 1) != odd) continue;
                    const uint32_t st = tile % CK_V_STAGES, slot = tile % CK_RAW_STAGES;
                    if (!(ok = wait(&sm.raw_full[slot], tile / CK_RAW_STAGES & 1))) break;
                    if (tile >= CK_V_STAGES && !(ok = wait(&sm.v_free[st], (tile / CK_V_STAGES - 1) & 1))) break;
                    const uint8_t *cp = sm.raw[slot] + from, *mp = sm.raw[slot] + meta_from;
                    const int base = sm.raw_base[slot][oct >> 1];
                    // tokens of the octet within the context, none without a page
                    const int valid = base < 0 ? 0 : min(8, max(0, share.ctx - base - 2 * pair0));
                    // a lane looks at one pair's scales or mins; tokens with a level, and NaN, take the long way
                    const __half2 most = ck_most(lds128(mp - 4 * g0 + 16 * (r & 3) + (r & 4 ? O4_VM - O4_VS : 0)));
                    const __half2 they = u32_as_h2(__shfl_xor_sync(0xffffffffu, h2_as_u32(most), 4));
                    const float2 z = r & 4 ? ck_sizes(they, most) : ck_sizes(most, they);
                    const float2 band = sm.share_band[(n_share - 1) % CK_SHARES];
                    const bool all = __all_sync(0xffffffffu, valid == 8 && fminf(z.x, z.y) >= band.x && z.x < band.y && z.y < band.y);
#pragma unroll 1
                    for (int g = 0; g < 2; ++g, cp += 4, mp += 4) {
                        uint32_t x[4][4];
                        if (all) {
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                const uint32_t s = lds32(mp + 16 * p), m = lds32(mp + 16 * p + (O4_VM - O4_VS));
                                __half2 c[4];
                                cc.codes(lds32(cp + 128 * p), c);
#pragma unroll
                                for (int n = 0; n < 4; ++n) x[n][p] = h2_as_u32(__hfma2(c[n], u32_as_h2(s), u32_as_h2(m)));
                            }
                        } else {
                            // in fp32; tokens past the context are 0, and so are those that hold what is not finite, whose logits
                            // the softmax makes NaN instead (a weight of 0 would not hide it from other rows; what else they hold,
                            // which has no level, is cut off at fp16's ends)
                            const int size = sm.share_size[(n_share - 1) % CK_SHARES];
                            const float2 level = make_float2(ck_pow2(-ck_level(ck_size(z.x, size))), ck_pow2(-ck_level(ck_size(z.y, size))));
#pragma unroll 1
                            for (int p = 0; p < 4; ++p) {
                                const uint32_t c = lds32(cp + 128 * p);
                                const float lo_f = __shfl_sync(0xffffffffu, level.x, (lane & 24) | p), hi_f = __shfl_sync(0xffffffffu, level.y, (lane & 24) | p);
                                const float2 s = __half22float2(u32_as_h2(lds32(mp + 16 * p))), m = __half22float2(u32_as_h2(lds32(mp + 16 * p + (O4_VM - O4_VS))));
                                const bool lo_ok = 2 * p < valid && isfinite(s.x) && isfinite(m.x), hi_ok = 2 * p + 1 < valid && isfinite(s.y) && isfinite(m.y);
#pragma unroll
                                for (int n = 0; n < 4; ++n) {
                                    const float lo = fmaf((float)(c >> (4 * n) & 15), s.x, m.x) * lo_f, hi = fmaf((float)(c >> (16 + 4 * n) & 15), s.y, m.y) * hi_f;
                                    const uint32_t y = pack_half2(lo_ok ? fminf(fmaxf(lo, -65504.f), 65504.f) : 0.f, hi_ok ? fminf(fmaxf(hi, -65504.f), 65504.f) : 0.f);
#pragma unroll
                                    for (int pp = 0; pp < 4; ++pp)
                                        if (pp == p) x[n][pp] = y;
                                }
                            }
                        }
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            *reinterpret_cast<uint4*>(sm.v[st] + to + (32 * g + 8 * n) * 128) = make_uint4(x[n][0], x[n][1], x[n][2], x[n][3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.raw_free[slot]);
                        mbar_arrive(&sm.v_full[st]);
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
        // ---- softmax of stream t: a thread a row
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, s_at = tmem + lanes + 128 * t, o_at = tmem + lanes + 256 + 128 * t;
        // 16 bytes of row x of the warp's
        auto q_slot = [&](int x, int y) { return sm.q[FEW ? 0 : t] + (32 * (warp & 3) + x) * 128 + (y >> 3) * (CK_QUERIES / 2) + (((y & 7) ^ (x & 7)) << 4); };
        uint32_t tile0 = 0, done = 0, parts = 0;
        bool ok = true;
        while (ok && next_share()) {
            const CkShare& g = sm.share[(n_share - 1) % CK_SHARES];
            const int two = g.two, n = g.n, ns = two ? n : (n + 1 - t) / 2;
            const int in_block = (two ? CK_ROW_TILE * t : 0) + row;
            const bool live = in_block < g.rows, idle = FEW && in_block - lane >= g.rows;
            const int in_seq = g.r0 + (live ? in_block : 0), pos = g.pos0 + in_seq / a.G;
            const int64_t at = (int64_t)g.h * a.n_tok * a.G + g.row0 + in_seq;  // the row among all
            // the row's queries: the last product with the ones before is done (FEW: of both streams)
            if (FEW && n_share > 1 && !(ok = wait(&sm.q_free, n_share & 1))) break;
            {
                const uint4* src = reinterpret_cast<const uint4*>(a.rot + (at - (live ? in_block : 0)) * D);  // of the block's first row
                // two rows at a time; FEW: four, half the channels each.  (All loads before the first store: one after the
                // other, each with L2's latency, they took 7 us of a block's start.)
                const int y = FEW ? 8 * t + (lane & 7) : lane & 15, x0 = FEW ? lane >> 3 : lane >> 4, rows = g.rows;
                uint4 q[FEW ? 8 : 16];
#pragma unroll
                for (int i = 0; i < (FEW ? 8 : 16); ++i) {
                    const int from = in_block - lane + x0 + (FEW ? 4 : 2) * i;
                    q[i] = __ldcg(src + (size_t)(from < rows ? from : 0) * (D / 8) + y);
                }
#pragma unroll
                for (int i = 0; i < (FEW ? 8 : 16); ++i) *reinterpret_cast<uint4*>(q_slot(x0 + (FEW ? 4 : 2) * i, y)) = q[i];
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.q_full[(n_share - 1) % CK_SHARES]);
            }
            const float f = __ldcg(a.row_scale + at);
            float ref = CK_NEG, l = 0.f;
            for (int x = 0; x < ns; ++x, ++done) {
                const uint32_t p_at = s_at + 64 * (done & 1);
                if (!(ok = wait(&sm.s_full[t][done & 1], done >> 1 & 1))) break;
                if (idle) {  // a warp without a row: whatever its lanes of P hold stays in them
                    if (lane == 0) mbar_arrive(&sm.p_full[t][done & 1]);
                    continue;
                }
                ck_fence_after();
                uint32_t p[32];
                const CkInfo& info = sm.info[(tile0 + (two ? x : 2 * x + t)) % CK_INFOS];
                const uint4 flags4 = lds128(info.flags);
                const uint32_t flags = flags4.x | flags4.y | flags4.z | flags4.w;
                const bool special = (info.special >> t & 1) | (flags & 1), levels = flags & 2;
                // 32 tokens, two pages: what the row does not see is -inf, what is not finite NaN; keys carried at 2^-4
                auto mask = [&](uint32_t* s, int c) {
#pragma unroll
                    for (int pg = 0; pg < 2; ++pg) {
                        const int base = info.base[2 * c + pg];
                        uint32_t see = base < 0 ? 0u : (1u << min(PAGE, max(0, pos - base + 1))) - 1u;
                        if (a.window) {
                            const int low = min(PAGE, max(0, pos - a.window + 1 - base)), sink = min(PAGE, max(0, a.sinks - base));
                            see &= ~((1u << low) - 1u) | ((1u << sink) - 1u);
                        }
                        const uint32_t marks = info.flags[2 * c + pg] & 1 ? info.marks[2 * c + pg] : 0u;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            if (marks >> (16 + i) & 1) s[16 * pg + i] = __float_as_uint(__uint_as_float(s[16 * pg + i]) * 16.f);
                            if (marks >> i & 1) s[16 * pg + i] = 0x7fffffffu;
                            if (!(see >> i & 1)) s[16 * pg + i] = 0xff800000u;
                        }
                    }
                };
                float weights;
                bool raise = x == 0;
                while (true) {  // (again, after the logits are read again, where a weight outgrew fp16)
                    uint32_t s[64];
                    ck_tmem_ld32(s, p_at);
                    ck_tmem_ld32(s + 32, p_at + 32);
                    ck_loaded32(s);
                    ck_loaded32(s + 32);
                    if (special) {
                        mask(s, 0);
                        mask(s + 32, 1);
                    }
                    if (raise) {  // the row's reference goes up to its largest product here, what it has so far down by as much
                        float top = -CUDART_INF_F;
#pragma unroll
                        for (int y = 0; y < 64; ++y) top = fmaxf(top, fmaf(__uint_as_float(s[y]), f, ck_size_f(info.z[y], info.share_bias)));
                        const float up = top > ref ? ceilf(top) : ref, c0 = ck_ex2(ref - up);
                        ref = up;
                        l *= c0;
                        if (x > 0) {
                            // the tile before is in the sums.  (Tiles take turns on two barriers: the parity then only has to tell it
                            // from the tile three before these logits, whose sums the logits of the tile before came after.)
                            if (!(ok = wait(&sm.o_done[t][(done - 1) & 1], (done - 1) >> 1 & 1))) break;
                            ck_fence_after();
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint32_t o[16];
                                ck_tmem_ld16(o, o_at + 16 * c);
                                ck_loaded16(o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * c0);
                                ck_tmem_st16(o, o_at + 16 * c);
                            }
                        }
                    }
                    const float off = CK_LIFT - ref;
                    float g = f;
                    if (levels) {  // the weights themselves; then the logits with levels
                        weights = 0.f;
                        g = 1.f;
#pragma unroll
                        for (int y = 0; y < 64; ++y) {
                            const float a = __uint_as_float(s[y]);
                            weights += ck_ex2(fmaf(a, f, off));
                            s[y] = __float_as_uint(fmaf(a, f, ck_level_f(ck_size_f(info.z[y], info.share_bias))));
                        }
                    }
                    const float2 g2 = make_float2(g, g), off2 = make_float2(off, off);
                    float2 sum[2];
                    sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float2 y = ck_fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), g2, off2);
                        y = make_float2(ck_ex2(y.x), ck_ex2(y.y));
                        sum[i & 1] = ck_add2(sum[i & 1], y);
                        p[i] = pack_half2(y.x, y.y);
                    }
                    sum[0] = ck_add2(sum[0], sum[1]);
                    const float carried = sum[0].x + sum[0].y;
                    if (!levels) weights = carried;
                    // (a sum that fp16 holds is one of weights that it holds)
                    if (raise || !__any_sync(0xffffffffu, carried > 65504.f)) break;
                    raise = true;
                }
                if (!ok) break;
                l += weights;
                ck_tmem_st32(p, p_at);  // (over logits that were read)
                ck_wait_st();
                ck_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[t][done & 1]);
            }
            tile0 += n;
            if (ok && ns > 0) {
                if (!(ok = wait(&sm.o_full[t], parts & 1))) break;
                ++parts;
                ck_fence_after();
                float* out = g.from > 0      ? a.extra + ((size_t)blockIdx.x * CK_ROWS + CK_ROW_TILE * t + row) * PART_STRIDE
                             : two || !t     ? a.main + (at + (live ? 0 : in_block)) * PART_STRIDE
                             : a.second_rows ? a.second + (((int64_t)g.b * a.H_kv + g.h) * a.second_rows + row) * PART_STRIDE
                                             : a.second + (at + (live ? 0 : in_block)) * PART_STRIDE;
                float m = ref - CK_LIFT, before = 0.f, now = 1.f;  // factors of the partial that stands there and of this run's
                if (g.again) {
                    const float2 ml = live ? __ldcg(reinterpret_cast<const float2*>(out)) : make_float2(m, 0.f);
                    const float top = fmaxf(m, ml.x);
                    before = ck_ex2(ml.x - top);
                    now = ck_ex2(m - top);
                    m = top;
                    l = fmaf(ml.y, before, l * now);
                }
                auto add = [&](uint32_t* o, const float* to, float before, float now) {  // (what this thread left there)
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(to));
                    o[0] = __float_as_uint(fmaf(y.x, before, __uint_as_float(o[0]) * now));
                    o[1] = __float_as_uint(fmaf(y.y, before, __uint_as_float(o[1]) * now));
                    o[2] = __float_as_uint(fmaf(y.z, before, __uint_as_float(o[2]) * now));
                    o[3] = __float_as_uint(fmaf(y.w, before, __uint_as_float(o[3]) * now));
                };
                if (live) *reinterpret_cast<float2*>(out) = make_float2(m, l);
                if constexpr (FEW) {
#pragma unroll 1
                    for (int c = 0; c < 4 && !idle; ++c) {
                        uint32_t o[32];
                        ck_tmem_ld32(o, o_at + 32 * c);
                        ck_loaded32(o);
                        if (live) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                if (g.again) add(o + i, out + 4 + 32 * c + i, before, now);
                                *reinterpret_cast<uint4*>(out + 4 + 32 * c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                            }
                        }
                    }
                } else {
                    // through the queries' place, which no product reads any more, so that a store covers two rows' 256 bytes
                    // (a row a lane, it touched 32 lines)
                    const int rows = g.rows - (in_block - lane);
                    out -= (int64_t)lane * PART_STRIDE;  // of the warp's first row
#pragma unroll 1
                    for (int c = 0; c < 2 && rows > 0; ++c) {
                        uint32_t o[64];
                        ck_tmem_ld32(o, o_at + 64 * c);
                        ck_tmem_ld32(o + 32, o_at + 64 * c + 32);
                        ck_loaded32(o);
                        ck_loaded32(o + 32);
#pragma unroll
                        for (int i = 0; i < 16; ++i) *reinterpret_cast<uint4*>(q_slot(lane, i)) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint4 v = lds128(q_slot(2 * i + (lane >> 4), lane & 15));
                            o[4 * i] = v.x, o[4 * i + 1] = v.y, o[4 * i + 2] = v.z, o[4 * i + 3] = v.w;
                        }
                        if (g.again) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int x = 2 * i + (lane >> 4);
                                const float before_x = __shfl_sync(0xffffffffu, before, x), now_x = __shfl_sync(0xffffffffu, now, x);
                                if (x < rows) add(o + 4 * i, out + (int64_t)x * PART_STRIDE + 4 + 64 * c + 4 * (lane & 15), before_x, now_x);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int x = 2 * i + (lane >> 4);
                            if (x < rows)
                                *reinterpret_cast<uint4*>(out + (int64_t)x * PART_STRIDE + 4 + 64 * c + 4 * (lane & 15)) =
                                    make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                        __syncwarp();
                    }
                }
                ck_fence_before();
            }
            if constexpr (FEW) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.q_free);
            }
        }
    }
    __syncwarp();
    ck_fence_before();
    __syncthreads();
    if (sm.dead && warp == CK_SOFTMAX + CK_UNPACK + 1)  // copies in flight land before the block ends
        for (uint32_t n = sm.stages, s = n > CK_RAW_STAGES ? n - CK_RAW_STAGES : 0; s < n; ++s)
            (void)mbar_wait_bounded(&sm.raw_full[s % CK_RAW_STAGES], (s / CK_RAW_STAGES) & 1, 1000000LL);
    if (warp == CK_SOFTMAX + CK_UNPACK) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ 3: finish

// CTAs of 256 threads take row tiles of a KV head, a warp 16 rows: their partials are merged in the layout of the A
// operand (a lane has eight times four values of two rows), normalised and rotated by R_v^T.  A 4K prompt of 32 heads: 43 us
// for 69 MB of partials and 34 of output (15 at the copy rate), bound by latency with two CTAs an SM.
__global__ void __launch_bounds__(256, 2) chunk_finish_kernel(const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    CkMatrix& R = *reinterpret_cast<CkMatrix*>(smem_raw);
    const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    // B: k = position of the unpacked values, n = output channel.  Lane t's four positions of a K step are 16 ks + 4 t and the
    // three after it: channels 32 (ks / 2) + 16 (t & 1) + 2 (ks & 1) + (t / 2), and 4, 8 and 12 further.  (Read before the
    // wait: the kernel that started this one did so after its own.)
    const float* Rv = a.Rv + (size_t)h * D * D;
#pragma unroll
    for (int y = threadIdx.x; y < D * 4 * 2; y += 256) {
        const int half = y & 1, g = (y >> 1) & 3, n = y >> 3;
        const float4* p = reinterpret_cast<const float4*>(Rv + (size_t)n * D + 32 * g + 16 * half);
        float k[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = __ldg(p + j);
            k[j][0] = v.x, k[j][1] = v.y, k[j][2] = v.z, k[j][3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            R.f[2 * g + (i >> 1)][n >> 3][(4 * (n & 7) + half + 2 * (i & 1)) ^ 8 * g] = make_uint2(pack_half2(k[0][i], k[1][i]), pack_half2(k[2][i], k[3][i]));
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int C = __ldcg(&a.plan->ctas), n_blocks = __ldcg(&a.plan->blocks);
    const int64_t total = __ldcg(&a.plan->total);
    // a warp at a time, its 16 rows of row tile x / 8
    for (int x = blockIdx.x * 8 + warp; x < 16 * n_blocks; x += gridDim.x * 8) {
        CkWalk w;
        w.e = x >> 4;
        w.read(a);
        const int two = w.k.rows > CK_ROW_TILE, i0 = 16 * (x & 15);  // in the block
        if (i0 >= w.k.rows) continue;
        const int wt = ck_weight(w.k.rows);
        const int64_t unit = w.k.start * a.H_kv + (int64_t)h * w.k.cost;
        // the share that holds the unit's first tile: a guess, put right by the cuts themselves
        int c = 0;
        if (w.k.tiles) {
            c = min(C - 1, (int)((float)unit / (float)total * (float)C));
            while (__ldcg(a.cut + c) > unit) --c;
            while (__ldcg(a.cut + c + 1) <= unit) ++c;
        }
        float M[2] = {CK_NEG, CK_NEG}, L[2] = {0.f, 0.f};
        float2 o[8][4];  // [K step][row, + 8; the next two positions]
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[ks][e] = make_float2(0.f, 0.f);
        const int ra = min(i0 + r, w.k.rows - 1), rb = min(i0 + r + 8, w.k.rows - 1);  // in the block
        const int64_t at = (int64_t)h * a.n_tok * a.G + (int64_t)w.k.q0 * a.G + w.k.r0;
        auto merge = [&](const float* base) {  // partials of the block's rows from base on
            const float* p[2] = {base + (int64_t)ra * PART_STRIDE, base + (int64_t)rb * PART_STRIDE};
            float keep[2], take[2];
            float2 y[8][4];
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float4 z = __ldcg(reinterpret_cast<const float4*>(p[e] + 4 + 16 * ks + 4 * t));
                    y[ks][e] = make_float2(z.x, z.y);
                    y[ks][e + 2] = make_float2(z.z, z.w);
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(p[e]));
                const float top = fmaxf(M[e], ml.x);
                keep[e] = ck_ex2(M[e] - top);
                take[e] = ck_ex2(ml.x - top);
                L[e] = fmaf(L[e], keep[e], ml.y * take[e]);
                M[e] = top;
            }
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[ks][e] = make_float2(fmaf(o[ks][e].x, keep[e & 1], y[ks][e].x * take[e & 1]), fmaf(o[ks][e].y, keep[e & 1], y[ks][e].y * take[e & 1]));
        };
#pragma unroll 1
        for (int from = 0, n; from < w.k.tiles; from += n, ++c) {
            n = min(w.k.tiles, ((int)min(__ldcg(a.cut + c + 1) - unit, (int64_t)w.k.cost) + wt - 1) / wt) - from;
            if (n <= 0) continue;
            const float* extra = a.extra + (size_t)c * CK_ROWS * PART_STRIDE;
#pragma unroll 1
            for (int s = 0; s < (two || n == 1 ? 1 : 2); ++s)  // (one row tile: a second stream, if there was a second tile)
                merge(from > 0         ? extra + (size_t)s * CK_ROW_TILE * PART_STRIDE
                      : !s            ? a.main + at * PART_STRIDE
                      : a.second_rows ? a.second + ((int64_t)w.k.b * a.H_kv + h) * a.second_rows * PART_STRIDE
                                      : a.second + at * PART_STRIDE);
        }
        uint32_t x16[8][4];
        float back[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float top = 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                top = fmaxf(fmaxf(top, fmaxf(fabsf(o[ks][e].x), fabsf(o[ks][e].y))), fmaxf(fabsf(o[ks][e + 2].x), fabsf(o[ks][e + 2].y)));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float sigma = ck_scale(top, 7);
            // (no token: 0; NaN stays NaN)
            back[e] = (L[e] > 0.f ? 1.f / L[e] : L[e] == L[e] ? 0.f : L[e]) / sigma;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                x16[ks][e] = pack_half2(o[ks][e].x * sigma, o[ks][e].y * sigma);
                x16[ks][e + 2] = pack_half2(o[ks][e + 2].x * sigma, o[ks][e + 2].y * sigma);
            }
        }
        __nv_bfloat16* out[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int in_seq = w.k.r0 + (e ? rb : ra);
            out[e] = a.out + ((int64_t)(w.k.q0 + in_seq / a.G) * a.H_q + (int64_t)h * a.G + in_seq % a.G) * D;
        }
#pragma unroll 1
        for (int nt = 0; nt < 16; nt += 4) {
            float c[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[j][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint2 b = R.f[ks][nt + j][lane ^ 8 * (ks >> 1)];
                    mma_f16_16816(c[j], x16[ks], b.x, b.y);
                }
            // a lane's two columns of four sets become eight of one: lane t gets set nt + t
            uint32_t z[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int j = 0; j < 4; ++j) z[e][j] = ck_pack(c[j][2 * e] * back[e], c[j][2 * e + 1] * back[e]);
#pragma unroll
                for (int k = 1; k < 4; k <<= 1) {  // transpose of the four lanes' four words
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (!(j & k)) {
                            const uint32_t send = t & k ? z[e][j] : z[e][j | k];
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, send, k);
                            if (t & k) z[e][j] = got;
                            else z[e][j | k] = got;
                        }
                }
                if (i0 + r + 8 * e < w.k.rows) *reinterpret_cast<uint4*>(out[e] + 8 * (nt + t)) = make_uint4(z[e][0], z[e][1], z[e][2], z[e][3]);
            }
        }
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

struct ChunkLayout {
    size_t plan, cut, block, scale, rot, main, second, extra, total;
    int max_blocks, block_rows;
    int64_t second_rows;
};
static ChunkLayout chunk_layout(int n_tok, int B, int H_q, int H_kv) {
    const int64_t G = H_q / H_kv, rows = (int64_t)n_tok * H_q, part = PART_STRIDE * 4;
    // Blocks of one row tile where a sequence has no more rows than that on the average.  Second streams: of blocks of one
    // row tile, of the others at most one per sequence
    ChunkLayout l;
    l.block_rows = (int64_t)n_tok * G <= (int64_t)B * CK_ROW_TILE ? CK_ROW_TILE : CK_ROWS;
    const bool few = l.block_rows == CK_ROWS && (int64_t)B * H_kv * CK_ROW_TILE < rows;
    l.max_blocks = (int)((int64_t)n_tok * G / l.block_rows + B);
    l.second_rows = few ? CK_ROW_TILE : 0;
    // (room for blocks of one row tile in either case: a workspace serves any call of fewer tokens or sequences)
    const size_t room = (size_t)((int64_t)n_tok * G / CK_ROW_TILE + B);
    l.plan = INT4_WS_BODY;
    l.cut = l.plan + 256;
    l.block = align_up(l.cut + (size_t)(kvq_device_sm_count() + 1) * 8, 256);
    l.scale = align_up(l.block + room * sizeof(CkBlock), 256);
    l.rot = align_up(l.scale + (size_t)rows * 4, 256);
    l.main = align_up(l.rot + (size_t)rows * D * 2, 256);
    l.second = align_up(l.main + (size_t)(rows * part), 256);
    l.extra = align_up(l.second + (size_t)((few ? (int64_t)B * H_kv * CK_ROW_TILE : rows) * part), 256);
    l.total = l.extra + (size_t)kvq_device_sm_count() * CK_ROWS * part;
    return l;
}

extern "C" size_t kvq_chunk_workspace_bytes(int n_tok, int B, int H_q, int H_kv) {
    kvq_status st;
    return chunk_refusal(n_tok, B, H_q, H_kv, st) ? 0 : chunk_layout(n_tok, B, H_q, H_kv).total;
}

// The shared memory opt-ins, once on each device.
static kvq_status chunk_smem_once() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    kvq_status st = kvq_check_cuda(cudaGetDevice(&dev), "kvq_chunk_attn_int4: cudaGetDevice");
    if (st != KVQ_OK) return st;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && done[dev]) return KVQ_OK;
    const struct {
        const void* fn;
        size_t bytes;
    } need[4] = {{(const void*)chunk_rotate_kernel, sizeof(CkRotate)},
                 {(const void*)chunk_stream_kernel<false>, sizeof(CkSmem<false>) + 1024},
                 {(const void*)chunk_stream_kernel<true>, sizeof(CkSmem<true>) + 1024},
                 {(const void*)chunk_finish_kernel, sizeof(CkMatrix)}};
    for (const auto& x : need) {
        st = kvq_check_cuda(cudaFuncSetAttribute(x.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)x.bytes),
                            "kvq_chunk_attn_int4 smem attribute");
        if (st != KVQ_OK) return st;
    }
    if (dev >= 0 && dev < 64) done[dev] = true;
    return KVQ_OK;
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
    const ChunkLayout l = chunk_layout(n_tok, B, H_q, H_kv);
    if (workspace_bytes < l.total)
        return kvq_set_error(KVQ_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, workspace_bytes, l.total);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
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
    a.window = window < (int64_t)max_pages_per_seq * PAGE ? window : 0;  // (a longer one holds every token)
    a.sinks = a.window ? sinks : 0;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.error = reinterpret_cast<uint32_t*>(ws);
    a.plan = reinterpret_cast<CkPlan*>(ws + l.plan);
    a.cut = reinterpret_cast<int64_t*>(ws + l.cut);
    a.block = reinterpret_cast<CkBlock*>(ws + l.block);
    a.max_blocks = l.max_blocks;
    a.block_rows = l.block_rows;
    a.row_scale = reinterpret_cast<float*>(ws + l.scale);
    a.rot = reinterpret_cast<__half*>(ws + l.rot);
    a.main = reinterpret_cast<float*>(ws + l.main);
    a.second = reinterpret_cast<float*>(ws + l.second);
    a.second_rows = l.second_rows;
    a.extra = reinterpret_cast<float*>(ws + l.extra);
    a.ctas = kvq_device_sm_count();
    a.drop = kvq_take_drop_next_copy();
    st = chunk_smem_once();
    if (st != KVQ_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int64_t row_tiles = ((int64_t)n_tok * a.G + CK_ROW_TILE - 1) / CK_ROW_TILE;
    auto capped = [&](int64_t want, int per_sm) { return (unsigned)std::min(want, std::max<int64_t>(1, per_sm * a.ctas / H_kv)); };  // CTAs per head
    st = kvq_check_cuda(launch_pdl(chunk_rotate_kernel, dim3(capped(row_tiles, 4) + 1, H_kv), dim3(256), sizeof(CkRotate), cs, a),
                        "kvq_chunk_attn_int4 rotate launch");
    if (st != KVQ_OK) return st;
    const bool one = l.block_rows == CK_ROW_TILE;
    st = kvq_check_cuda(launch_pdl(one ? chunk_stream_kernel<true> : chunk_stream_kernel<false>, dim3(a.ctas), dim3(CK_THREADS),
                                   (one ? sizeof(CkSmem<true>) : sizeof(CkSmem<false>)) + 1024, cs, a),
                        "kvq_chunk_attn_int4 launch");
    if (st != KVQ_OK) return st;
    return kvq_check_cuda(launch_pdl(chunk_finish_kernel, dim3(capped(2 * (int64_t)l.max_blocks, 4), H_kv), dim3(256), sizeof(CkMatrix), cs, a),
                          "kvq_chunk_attn_int4 finish launch");
}
