// Choice of key blocks for block-sparse attention: the score of query block i
// and key block j of one head is the dot product of their mean query and mean
// key, and each query block keeps the topk best-scored key blocks.
//
// The choice is a comparison of scores that lie close together (among a few
// hundred scores of a row, neighbours 1e-6 apart are a matter of course), so it
// is made on scores in 64 bits: it depends on the inputs alone, not on the order
// of additions.  Computing them all in fp64 would cost more than reading q and k
// (190 us against 62 us at the 480p pair's 24 x 336 x 624 scores), so rows of up
// to 2048 blocks go in two stages:
//   block_mean_kernel   one pass over q and k: fp64 means, the same scaled to unit
//                       length in fp16, and their norms;
//   block_score_kernel  unit products on the tensor cores times the key's norm:
//                       within SCORE_ERROR |k| of the 64-bit score over |q|;
//   block_topk_kernel   the topk-th best of a row, from a first place by the row's mean
//                       and spread through interpolation (bisection where that does
//                       not settle it); only blocks that the error lets lie on either
//                       side of the border (seven or so of several hundred) are scored
//                       again, in fp64, and ranked by that.
// (With hi + lo parts and three products fewer are scored again, but the products
// and their operands cost more than that saves: 30 against 14 us of the pair's.)
// Longer rows: block_score64_kernel and block_topk64_kernel, all in fp64.
//
// Measured, us: means 75 (5.4 TB/s), scores 14, top-k 28 of the 480p pair (B = 2, 12
// heads, 32760 tokens, 336 x 624 blocks); 248 (6.3 TB/s), 44 and 93 with 40 heads, 75600
// tokens, 720 x 720 blocks and a mask.  The larger case's means run at the rate of a copy;
// the pair's are held by the conversions to fp64 (74 % of their pipe) as much as by memory
// (66 % of DRAM's peak), in many short CTAs; the scores are bound by
// their way through the L2, and 64 x 128 tiles, which read a quarter less, take 2 us off
// the 44; the top-k by instruction issue (65 %): 2300 per row of 720.  Starting each kernel
// while the one before it drains costs the large cases more (1 %) than it saves.
// A NaN or an infinity in a head's keys leaves no bound for its rows: all their scores are
// taken in fp64 by block_topk_kernel, a warp per row.  With one in every head 355 us for 122
// (pair), 2590 for 394 (40 heads).
#include <cuda_fp16.h>

#include <cfloat>
#include <climits>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace wan {

namespace {

constexpr int SCORE_Q = 32, SCORE_K = 64;  // fp64 score kernel: query x key blocks per CTA
constexpr int K_PITCH = 129;               // doubles per staged mean (odd: column reads hit all banks)
constexpr int MAX_FAST = 2048;             // key blocks of the two-stage path
// Bound of a unit product's error: an fp16 rounding is off by 2^-11 of the element
// (or by 2^-25 where it is subnormal), on either side: 2 * 2^-11 (1 + 2^-11) + 2 *
// 2^-25 * sqrt(128); 128 fp32 additions, truncated, add at most 128 * 2^-23.
constexpr float SCORE_ERROR = 1.007e-3f;
constexpr float SCORE_TINY = 1e-36f;            // below it scores lose bits to underflow

// Means of the blocks of q (first g.q_blocks() CTAs) and k, per head: fp64, fp16 of
// unit length, and norm (NaN or infinite where a mean is).  One CTA per block and
// column slice, eight columns per thread, four tokens loaded (evict-first: nothing
// reads them again here; 6 us of the pair's 81) while the four before are added; where
// there are few CTAs (a small grid) RG = 4 groups of threads take every fourth eight
// tokens each: a block is a chain of loads (14.5 -> 7.6 us at 15 blocks).  Every token
// is added in fp64: it must not matter what stands beside a small one.  (Sums of
// four tokens in fp32 first, which lose a value 2^17 times smaller than its
// neighbour, take 2 us less of the pair's; the same with the rounding errors
// kept beside them 60 more.)
struct MeanOut {
    double* mean;           // [B, heads, blocks, 128]
    __half* unit;           // [B, heads, blocks, 128], null: not wanted
    float* norm;            // [B, heads, norm_pitch]
    int norm_pitch;
};
template <int RG>
__global__ void __launch_bounds__(256) block_mean_kernel(const __nv_bfloat16* __restrict__ q, long long ldq,
                                                         const __nv_bfloat16* __restrict__ k, long long ldk, int heads,
                                                         const __grid_constant__ BlockGrid g, const MeanOut oq,
                                                         const MeanOut ok) {
    __shared__ int tokens[128];
    const int b = blockIdx.z;
    const bool keys = blockIdx.x >= g.q_blocks();
    const int blk = keys ? blockIdx.x - g.q_blocks() : blockIdx.x;
    const int* dim = keys ? g.k : g.q;
    const int* box = keys ? g.kb : g.qb;
    const int F = dim[0], H = dim[1], W = dim[2];
    const int nH = (H + box[1] - 1) / box[1], nW = (W + box[2] - 1) / box[2], nF = (F + box[0] - 1) / box[0];
    const int f0 = blk / (nH * nW) * box[0], i0 = blk / nW % nH * box[1], j0 = blk % nW * box[2];
    const int ef = min(box[0], F - f0), ei = min(box[1], H - i0), ej = min(box[2], W - j0);
    const int n = ef * ei * ej;
    const int y = RG > 1 ? threadIdx.y : 0;
    for (int t = y * blockDim.x + threadIdx.x; t < n; t += RG * blockDim.x)
        tokens[t] = ((f0 + t / (ej * ei)) * H + i0 + t / ej % ei) * W + j0 + t % ej;
    __syncthreads();
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    const bool mine = col < heads * 128;  // whole heads (16 threads) at a time
    const long long ld = keys ? ldk : ldq;
    const __nv_bfloat16* base = (keys ? k : q) + (long long)b * F * H * W * ld + (mine ? col : 0);
    double acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = 0.0;
    auto add = [&](const uint4 (&v)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 p = unpack_bf16(w[c]);
                acc[2 * c] += (double)p.x;
                acc[2 * c + 1] += (double)p.y;
            }
        }
    };
    auto fetch = [&](int t, uint4 (&v)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] = t + u < n ? __ldcs(reinterpret_cast<const uint4*>(base + (long long)tokens[t + u] * ld)) : make_uint4(0, 0, 0, 0);
    };
    if (RG == 1) {
        uint4 a[4], b[4];  // past the end fetch() gives zeros
        fetch(0, a);
        for (int t = 0; t < n; t += 8) {
            fetch(t + 4, b);
            add(a);
            fetch(t + 8, a);
            add(b);
        }
    } else {
        for (int t = y * 8; t < n; t += 8 * RG) {
            uint4 a[4], b[4];
            fetch(t, a);
            fetch(t + 4, b);
            add(a);
            add(b);
        }
    }
    if constexpr (RG > 1) {
        __shared__ double part[RG - 1][8][64];
        if (y > 0) {
#pragma unroll
            for (int c = 0; c < 8; ++c) part[y - 1][c][threadIdx.x] = acc[c];
        }
        __syncthreads();
        if (y > 0) return;
#pragma unroll
        for (int r = 0; r < RG - 1; ++r)
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] += part[r][c][threadIdx.x];
    }
    const MeanOut& o = keys ? ok : oq;
    const long long at = ((long long)b * heads + (mine ? col / 128 : 0)) * (nF * nH * nW) + blk;
    // a whole block's count is a power of two: the same numbers without eight divisions
    if ((n & (n - 1)) == 0) {
        const double part = 1.0 / (double)n;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] *= part;
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] /= (double)n;
    }
    double ss = 0.0;
#pragma unroll
    for (int c = 0; c < 8; ++c) ss += acc[c] * acc[c];
    if (o.unit) {
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
    }
    if (!mine) return;
    double* dst = o.mean + at * 128 + col % 128;
#pragma unroll
    for (int c = 0; c < 8; c += 2) *reinterpret_cast<double2*>(dst + c) = make_double2(acc[c], acc[c + 1]);
    if (!o.unit) return;
    const double norm = sqrt(ss);
    const double inv = norm > 0.0 && norm < 1e300 ? 1.0 / norm : 0.0;
    uint32_t u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const __half2 h = __floats2half2_rn((float)(acc[2 * c] * inv), (float)(acc[2 * c + 1] * inv));
        u[c] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(o.unit + at * 128 + col % 128) = make_uint4(u[0], u[1], u[2], u[3]);
    if ((threadIdx.x & 15) == 0) o.norm[((long long)b * heads + col / 128) * o.norm_pitch + blk] = (float)norm;
}

// ---------------------------------------------------------------- two-stage path
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// scores[bh][i][j] = (unit mean of q block i) . (unit mean of k block j) * |k j|,
// rows `pitch` apart and filled up with -inf.  64 x 64 scores per CTA, four warps of 32 x 32; both operands
// whole (K = 128) in shared memory, 256 bytes a row, 16-byte pieces swizzled by the
// row.  mma.sync and not tcgen05: a few microseconds of work, in tiles too small
// for a 128-row accumulator.
constexpr int ST = 64;
__global__ void __launch_bounds__(128) block_score_kernel(const __half* __restrict__ qu, const __half* __restrict__ ku,
                                                          const float* __restrict__ kn, int nq, int nk, int pitch,
                                                          float* __restrict__ scores) {
    __shared__ uint4 tile[2 * ST * 16];
    const int q0 = blockIdx.y * ST, k0 = blockIdx.x * ST;
    const long long bh = blockIdx.z;
#pragma unroll
    for (int i = threadIdx.x; i < 2 * ST * 16; i += 128) {
        const int which = i / (ST * 16), r = i / 16 % ST, c = i % 16;
        const int at = (which ? k0 : q0) + r, n = which ? nk : nq;
        const __half* src = (which ? ku : qu) + (bh * n + at) * 128 + c * 8;
        tile[(which * ST + r) * 16 + (c ^ (r & 7))] = at < n ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m0 = (warp >> 1) * 32, n0 = (warp & 1) * 32;
    const uint32_t sq = smem_u32(tile), sk = sq + ST * 256;
    float acc[2][4][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][j][c] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        // 8 x 8 matrices of an x4 load: A rows lane & 15, pieces 2 kk + (lane >> 4); B two n8 tiles
        uint32_t a[2][4], b[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ra = m0 + 16 * i + (lane & 15), ca = 2 * kk + (lane >> 4);
            ldmatrix4(a[i], sq + ra * 256 + ((ca ^ (ra & 7)) << 4));
            const int rb = n0 + 16 * i + (lane & 7) + ((lane >> 4) << 3), cb = 2 * kk + ((lane >> 3) & 1);
            ldmatrix4(b[i], sk + rb * 256 + ((cb ^ (rb & 7)) << 4));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_16816(acc[i][j], a[i], b[j >> 1][(j & 1) * 2], b[j >> 1][(j & 1) * 2 + 1]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = k0 + n0 + 8 * j + (lane & 3) * 2;  // even, as the pitch is
        if (col >= pitch) continue;
        const float s0 = col < nk ? __ldg(kn + bh * pitch + col) : 0.f, s1 = col + 1 < nk ? __ldg(kn + bh * pitch + col + 1) : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = q0 + m0 + 16 * i + half * 8 + (lane >> 2);
                if (row < nq)
                    *reinterpret_cast<float2*>(scores + (bh * nq + row) * pitch + col) =
                        make_float2(col < nk ? acc[i][j][half * 2] * s0 : -INFINITY,
                                    col + 1 < nk ? acc[i][j][half * 2 + 1] * s1 : -INFINITY);
            }
    }
}

// A score as a 64-bit key in the same order: NaN ranks with -inf, keys of
// allowed blocks are above 0 and below ~0.
__device__ __forceinline__ unsigned long long score_key(double s) {
    if (!(s == s)) s = -INFINITY;
    if (s == 0.0) s = 0.0;  // -0 and 0 tie
    const unsigned long long u = (unsigned long long)__double_as_longlong(s);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// A key of the fp32 scores in their order: 0 is free for forbidden blocks, ~0 for
// those asked for.
__device__ __forceinline__ uint32_t score_key32(float s) {
    if (!(s == s)) s = -INFINITY;
    const uint32_t u = __float_as_uint(s);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key32_score(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }

// keys[bh][i][j] = key of (q mean i) . (k mean j); 0 where the mask forbids the
// block, ~0 where it asks for it.  Each thread 8 query x 2 key blocks.
__global__ void __launch_bounds__(128) block_score64_kernel(const double* __restrict__ qm, const double* __restrict__ km,
                                                          const uint8_t* __restrict__ mask, int nq, int nk,
                                                          unsigned long long* __restrict__ keys) {
    extern __shared__ double sm[];
    double* sq = sm;                        // [128][SCORE_Q]: dimension-major
    double* sk = sm + 128 * SCORE_Q;        // [SCORE_K][K_PITCH]
    const int q0 = blockIdx.y * SCORE_Q, k0 = blockIdx.x * SCORE_K;
    const double* q = qm + (long long)blockIdx.z * nq * 128;
    const double* k = km + (long long)blockIdx.z * nk * 128;
    for (int i = threadIdx.x; i < SCORE_Q * 128; i += 128) {
        const int r = i & (SCORE_Q - 1), d = i / SCORE_Q;
        sq[d * SCORE_Q + r] = q0 + r < nq ? q[(long long)(q0 + r) * 128 + d] : 0.0;
    }
    for (int i = threadIdx.x; i < SCORE_K * 128; i += 128) {
        const int r = i >> 7, d = i & 127;
        sk[r * K_PITCH + d] = k0 + r < nk ? k[(long long)(k0 + r) * 128 + d] : 0.0;
    }
    __syncthreads();
    const int c = threadIdx.x & 31, rg = (threadIdx.x >> 5) * 8;
    double a0[8], a1[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) a0[r] = a1[r] = 0.0;
    const double* kc0 = sk + c * K_PITCH;
    const double* kc1 = sk + (c + 32) * K_PITCH;
#pragma unroll 4
    for (int d = 0; d < 128; ++d) {
        const double k0v = kc0[d], k1v = kc1[d];
        const double2* qr = reinterpret_cast<const double2*>(sq + d * SCORE_Q + rg);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const double2 v = qr[r];
            a0[2 * r] = fma(v.x, k0v, a0[2 * r]);
            a0[2 * r + 1] = fma(v.y, k0v, a0[2 * r + 1]);
            a1[2 * r] = fma(v.x, k1v, a1[2 * r]);
            a1[2 * r + 1] = fma(v.y, k1v, a1[2 * r + 1]);
        }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int i = q0 + rg + r;
        if (i >= nq) break;
        unsigned long long* row = keys + ((long long)blockIdx.z * nq + i) * nk;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int j = k0 + c + half * 32;
            if (j >= nk) continue;
            unsigned long long key = score_key(half ? a1[r] : a0[r]);
            if (mask) {
                const uint8_t m = __ldg(mask + (long long)i * nk + j);
                key = m == 0 ? 0ull : m == 1 ? key : ~0ull;
            }
            row[j] = key;
        }
    }
}

// The topk best blocks of a row: one warp per row, a lane holding the scores of NPL
// consecutive blocks in registers (nk <= 32 NPL).  A threshold `at` that leaves
// topk scores is found by interpolation (half a dozen counts).  With d the bound of
// all scores' errors, topk blocks have 64-bit scores of at - d or more, and the blocks
// below the threshold less than at + d: a block whose score lies more than 2 d above
// the threshold is taken, one more than 2 d below is not, and the close ones in
// between (twenty or so of several hundred, where blocks of fewer tokens at the
// grid's edge have longer means), one per lane, are narrowed by their own bounds d_j:
// taken is a_j - d_j > U = max (a_j + d_j) over the topk-th best score and all below
// it, left is a_j + d_j < L = min (a_j - d_j) over the topk best.  What remains (seven
// or so) is ranked by its fp64 scores, equal ones to the lower block.
struct TopkParams {
    const float* scores;            // [B heads nq, pitch]
    const double *qm, *km;          // means
    const float *qn, *kn;           // their norms: [B heads, nq], [B heads, pitch]
    const uint8_t* mask;            // [nq, nk] or null
    unsigned long long* exact;      // [rows, nk]: used by rows with many close scores only
    int nq, nk, pitch, topk;
    int *blocks, *counts;
};
// Up to 24 scores per lane seven CTAs share an SM, at 72 registers (eight, at 64, spill: 117
// against 114 us for the pair's three kernels; six: 118).  The scans are unrolled over NPL, so
// their cost is NPL's, not the row's: it is the next multiple of 4 up to 32 and of 16 beyond.
// All three kernels of 336 x 800 blocks with NPL 28 against 32: 44 against 48 us; 336 x 1200
// and 1500 with 48 against 64: 72 against 79 and 80 against 93; 336 x 200 with 8 against 12:
// 25 against 26.
template <int NPL>
__global__ void __launch_bounds__(128, NPL <= 24 ? 7 : 1) block_topk_kernel(const __grid_constant__ TopkParams p) {
    using Bits = typename std::conditional<(NPL > 32), unsigned long long, uint32_t>::type;
    // rows come in coalesced and are read back a lane's consecutive blocks at a time
    __shared__ int again[4][32];
    __shared__ uint32_t longest[4];
    __shared__ float4 stage[4][NPL * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nk = p.nk, j0 = lane * NPL;  // the lane's first block
    const long long bh = blockIdx.y;
    const int i_q = blockIdx.x * 4 + warp;
    const long long row = bh * p.nq + i_q;
    const float* kn = p.kn + bh * p.pitch;
    uint32_t most = 0;  // the head's longest key, as bits: NaN above infinity above all numbers
    for (int i = threadIdx.x; i < nk; i += 128) most = max(most, __float_as_uint(__ldg(kn + i)) & 0x7fffffffu);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) longest[warp] = most;
    if (i_q < p.nq) {
        const float4* src = reinterpret_cast<const float4*>(p.scores + row * p.pitch);
#pragma unroll
        for (int i = 0; i < NPL / 4; ++i)
            stage[warp][i * 32 + lane] = i * 32 + lane < p.pitch / 4
                                             ? __ldg(src + i * 32 + lane)
                                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    __syncthreads();
    if (i_q >= p.nq) return;
    const float key_norm = __uint_as_float(max(max(longest[0], longest[1]), max(longest[2], longest[3])));
    const bool number = key_norm < 1e38f && p.qn[row] < INFINITY;  // every score is one
    // scores, -inf where there is no block or it is not the score that decides: `extra` are the
    // blocks asked for, `allowed` those left to their scores
    float f[NPL];
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
        const float4 v = stage[warp][(j0 + i) / 4];
        f[i] = v.x;
        f[i + 1] = v.y;
        f[i + 2] = v.z;
        f[i + 3] = v.w;
    }
    // their mean and spread, from the lanes that are full (before the mask: a guess)
    float sum = 0.f, sum2 = 0.f;
    {
        uint64_t a = 0ull, b = 0ull;
#pragma unroll
        for (int i = 0; i < NPL; i += 2) {
            const uint64_t x = f2pack(f[i], f[i + 1]);
            a = add2(a, x);
            b = fma2(x, x, b);
        }
        float x, y;
        f2unpack(a, x, y);
        sum = x + y;
        f2unpack(b, x, y);
        sum2 = x + y;
    }
    const bool full = fabsf(sum) < INFINITY && sum2 < INFINITY;
    const float seen = NPL * __popc(__ballot_sync(0xffffffffu, full));
    if (!full) sum = sum2 = 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum2 += __shfl_xor_sync(0xffffffffu, sum2, o);
    }
    const int here = min(max(nk - j0, 0), NPL);
    Bits allowed = here == 0 ? Bits(0) : ~Bits(0) >> (sizeof(Bits) * 8 - here), extra = 0;
    if (p.mask) {
        // the lane's bytes as words, shifted into place; a word is read if a byte of the row is in it
        const uintptr_t first = reinterpret_cast<uintptr_t>(p.mask) + (long long)i_q * nk + j0;
        const uintptr_t end = reinterpret_cast<uintptr_t>(p.mask) + ((long long)i_q + 1) * nk;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(first & ~uintptr_t(3));
        const uint32_t shift = (uint32_t)(first & 3) * 8;
        Bits by_score = 0;
        uint32_t low = first < end ? __ldg(words) : 0u;
#pragma unroll
        for (int i = 0; i < NPL; i += 4) {
            const uint32_t high = reinterpret_cast<uintptr_t>(words + i / 4 + 1) < end ? __ldg(words + i / 4 + 1) : 0u;
            const uint32_t m = __funnelshift_r(low, high, shift);
            low = high;
            // bytes above 1 and bytes that are 1, each as one bit, gathered by a multiplication
            const uint32_t z = m & 0xfefefefeu, ahead = ((((z & 0x7f7f7f7fu) + 0x7f7f7f7fu) | z) >> 7) & 0x01010101u;
            by_score |= (Bits)(((m & ~ahead & 0x01010101u) * 0x01020408u) >> 24 & 15u) << i;
            extra |= (Bits)((ahead * 0x01020408u) >> 24 & 15u) << i;
        }
        extra &= allowed;
        allowed &= by_score;
#pragma unroll
        for (int i = 0; i < NPL; ++i) f[i] = allowed >> i & 1 ? f[i] : -INFINITY;
    }
    auto bits_of = [](Bits x) { return NPL > 32 ? __popcll(x) : __popc((uint32_t)x); };
    auto count = [&](float at) {  // scores >= at
        int n = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) n += f[i] >= at;
        return (int)__reduce_add_sync(0xffffffffu, n);
    };
    const int always = p.mask ? __reduce_add_sync(0xffffffffu, bits_of(extra)) : 0;
    const int scored = p.mask ? __reduce_add_sync(0xffffffffu, bits_of(allowed)) : nk;
    const int take = min(p.topk, always + scored);
    const int want = take - always;  // of the scored ones
    int* dst = p.blocks + row * p.topk;
    // set bits of the lanes before
    auto before = [&](Bits bits) {
        const int mine = bits_of(bits);
        int n = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += v;
        }
        return n - mine;
    };
    // the picks to their places, ascending
    auto put = [&](Bits picks) {
        int to = before(picks);
        while (picks) {
            const int i = NPL > 32 ? __ffsll((long long)picks) - 1 : __ffs((int)picks) - 1;
            picks &= picks - 1;
            dst[to++] = j0 + i;
        }
        for (int i = take + lane; i < p.topk; i += 32) dst[i] = -1;
        if (lane == 0) p.counts[row] = take;
    };
    // picks among equals: the first `left` of the set bits, lanes in order
    auto first_of = [&](Bits bits, int left) -> Bits {
        Bits out = 0;
        for (int n = before(bits); bits && n < left; ++n) {
            const Bits low = bits & (~bits + 1);
            out |= low;
            bits ^= low;
        }
        return out;
    };
    if (want <= 0) {  // blocks asked for alone, the lowest of them
        put(first_of(extra, take));
        return;
    }
    if (want == scored) {  // all that is allowed
        put(extra | allowed);
        return;
    }
    Bits sure = extra, close = allowed;  // all are close where a mean is not finite
    float at = -FLT_MAX;
    if (number) {
        // at: a score that `want` scores reach, and no more unless equal ones lie at the border.
        // The first place is where normally distributed scores would have it, the next is a
        // step by their density there, and between two that enclose it the counts lead, every
        // third time half way (five counts for a normal row); where that does not settle it
        // (scores of many magnitudes) half way between the scores' bit patterns.
        const float mean = sum / seen, spread = sqrtf(fmaxf(sum2 / seen - mean * mean, 0.f));
        const float share = (float)want / (float)scored;
        // the logistic curve of slope 1.702 is near the normal one
        float mid = mean + spread * 0.4073f * log2f((1.f - share) / share);
        const float per_count = spread / (1.702f * (float)want * (1.f - share));
        float lo = -FLT_MAX, hi = FLT_MAX;
        int n_at = scored, n_hi = 0;  // scores >= lo; >= the last place that was too high
        for (int step = 0; n_at != want && lo < hi; ++step) {
            if (step >= 24 || !(mid > lo && mid <= hi)) {
                const uint32_t a = score_key32(lo), b = score_key32(hi);
                mid = key32_score(a + ((b - a) >> 1) + 1);
            }
            const int n = count(mid);
            const float tried = mid;
            if (n >= want) {
                lo = at = mid;
                n_at = n;
            } else {
                hi = key32_score(score_key32(mid) - 1);  // the next lower float
                n_hi = n;
            }
            if (lo > -FLT_MAX && hi < FLT_MAX)
                mid = lo + (step % 3 == 2 ? 0.5f : fminf(fmaxf((float)(n_at - want) / (float)(n_at - n_hi), 0.05f), 0.95f)) * (hi - lo);
            else
                mid = tried + ((float)(n - want) + (n >= want ? 1.f : -1.f)) * per_count * (float)(1 << min(step, 8));
        }
        const float d2 = 2.f * fmaf(SCORE_ERROR, key_norm, SCORE_TINY), above = at + d2, below = at - d2;
        close = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            sure |= (Bits)(f[i] > above) << i;
            close |= (Bits)(f[i] >= below) << i;
        }
        close &= allowed & ~sure;
        if (__reduce_add_sync(0xffffffffu, bits_of(close)) > 32) {
            float L = INFINITY, U = -INFINITY, vk = INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) vk = fminf(vk, f[i] >= at ? f[i] : INFINITY);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) vk = fminf(vk, __shfl_xor_sync(0xffffffffu, vk, o));
            auto bound = [&](int i) { return fmaf(SCORE_ERROR, j0 + i < nk ? __ldg(kn + j0 + i) : 0.f, SCORE_TINY); };
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const float d = bound(i);
                L = fminf(L, f[i] >= at ? f[i] - d : INFINITY);
                U = fmaxf(U, f[i] <= vk ? f[i] + d : -INFINITY);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                L = fminf(L, __shfl_xor_sync(0xffffffffu, L, o));
                U = fmaxf(U, __shfl_xor_sync(0xffffffffu, U, o));
            }
            sure = extra;
            close = 0;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const float d = bound(i);
                sure |= (Bits)(f[i] - d > U) << i;
                close |= (Bits)(f[i] + d >= L) << i;
            }
            close &= allowed & ~sure;
        }
    }
    const int n_sure = __reduce_add_sync(0xffffffffu, bits_of(sure));
    const int n_close = __reduce_add_sync(0xffffffffu, bits_of(close));
    const int need = take - n_sure;
    if (n_close == need) {
        put(sure | close);
        return;
    }
    // fp64 keys: eight lanes per block, four blocks at a time; every lane gets its group's
    const int sub = lane & 7;
    const double2* qd = reinterpret_cast<const double2*>(p.qm + row * 128) + sub;
    auto exact_key = [&](int j) {
        const double2* kd = reinterpret_cast<const double2*>(p.km + (bh * nk + j) * 128) + sub;
        double2 kv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) kv[i] = __ldg(kd + 8 * i);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double2 qv = __ldg(qd + 8 * i);
            s = fma(qv.y, kv[i].y, fma(qv.x, kv[i].x, s));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return score_key(s);
    };
    if (n_close <= 32) {
        // lane n has the n-th close block
        const int first = before(close);
        Bits rest = close;
        for (int n = first; rest; ++n) {
            const Bits low = rest & (~rest + 1);
            again[warp][n] = j0 + bits_of(low - 1);
            rest ^= low;
        }
        __syncwarp();
        bool in = false, open = lane < n_close;
        int left = need;
        if (number) {
            // their own bounds leave fewer: L and U as above, which no other block decides
            const int j = again[warp][open ? lane : 0];
            const float a = reinterpret_cast<const float*>(stage[warp])[j];
            const float d = fmaf(SCORE_ERROR, __ldg(kn + j), SCORE_TINY);
            const uint32_t none = 0xffffffffu;
            const uint32_t vk = __reduce_min_sync(none, open && a >= at ? score_key32(a) : none);
            const float L = key32_score(__reduce_min_sync(none, open && a >= at ? score_key32(a - d) : none));
            const float U = key32_score(__reduce_max_sync(none, open && score_key32(a) <= vk ? score_key32(a + d) : 0u));
            in = open && a - d > U;
            open = open && !in && a + d >= L;
            left -= __popc(__ballot_sync(none, in));
            const unsigned still = __ballot_sync(none, open);
            __syncwarp();  // the list has been read
            if (open) again[warp][__popc(still & ((1u << lane) - 1))] = j;
            __syncwarp();
        }
        // lane n ranks the n-th block that is left among all of them
        const unsigned still = __ballot_sync(0xffffffffu, open);
        const int n_open = __popc(still);
        unsigned chosen = __ballot_sync(0xffffffffu, in);
        if (n_open == left) {
            chosen |= still;
        } else {
            unsigned long long k = 0;
#pragma unroll 1
            for (int c = 0; c < n_open; c += 4) {
                const unsigned long long e = exact_key(again[warp][min(c + (lane >> 3), n_open - 1)]);
                const unsigned long long got = __shfl_sync(0xffffffffu, e, (lane & 3) * 8);
                if (lane >= c && lane < c + 4) k = got;  // c is a multiple of 4: lane & 3 == lane - c
            }
            int better = 0;
            for (int l = 0; l < n_open; ++l) {
                const unsigned long long other = __shfl_sync(0xffffffffu, k, l);
                better += other > k || (other == k && l < lane);
            }
            const unsigned best = __ballot_sync(0xffffffffu, lane < n_open && better < left);
            const int mine = __popc(still & ((1u << lane) - 1));  // the lane's own block's place among those left
            chosen |= __ballot_sync(0xffffffffu, open && (best >> mine & 1));
        }
        rest = close;
        for (int n = first; rest; ++n) {
            const Bits low = rest & (~rest + 1);
            if (chosen >> n & 1) sure |= low;
            rest ^= low;
        }
        put(sure);
        return;
    }
    // many close scores (equal blocks, infinities): fp64 keys through memory
    unsigned long long* ek = p.exact + row * nk;
    unsigned long long lo64 = ~0ull, hi64 = 0;
#pragma unroll 1
    for (int c = 0; c < nk; c += 4) {
        const int j = min(c + (lane >> 3), nk - 1);
        const unsigned long long e = exact_key(j);
        if (sub == 0) ek[j] = e;
    }
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < NPL; ++i)
        if (close >> i & 1) {
            lo64 = min(lo64, ek[j0 + i]);
            hi64 = max(hi64, ek[j0 + i]);
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo64 = min(lo64, __shfl_xor_sync(0xffffffffu, lo64, o));
        hi64 = max(hi64, __shfl_xor_sync(0xffffffffu, hi64, o));
    }
    auto reach64 = [&](unsigned long long v) -> Bits {  // close blocks with keys >= v
        Bits bits = 0;
#pragma unroll 1
        for (int i = 0; i < NPL; ++i)
            if (close >> i & 1) bits |= (Bits)(ek[j0 + i] >= v) << i;
        return bits;
    };
    auto count64 = [&](unsigned long long v) { return (int)__reduce_add_sync(0xffffffffu, bits_of(reach64(v))); };
    unsigned long long at64 = lo64;
    int n64 = n_close;
    while (n64 != need && lo64 < hi64) {
        const unsigned long long mid = lo64 + ((hi64 - lo64) >> 1) + 1;
        const int n = count64(mid);
        if (n >= need) {
            lo64 = mid;
            at64 = mid;
            n64 = n;
        } else {
            hi64 = mid - 1;
        }
    }
    if (n64 == need) {
        put(sure | reach64(at64));
    } else {  // equal scores at the border: the lower blocks
        const Bits above = reach64(at64 + 1), equal = reach64(at64) & ~above;
        const int n_above = __reduce_add_sync(0xffffffffu, bits_of(above));
        put(sure | above | first_of(equal, need - n_above));
    }
}

// Longer rows: one CTA per row, fp64 keys in shared memory, bisected the same way.
__global__ void __launch_bounds__(256) block_topk64_kernel(const unsigned long long* __restrict__ keys, int nk, int topk,
                                                             int* __restrict__ blocks, int* __restrict__ counts) {
    extern __shared__ unsigned long long key[];
    __shared__ int sums[8];
    __shared__ unsigned long long ends[16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const unsigned long long* src = keys + row * nk;
    unsigned long long lo = ~0ull, hi = 0;
    for (int i = tid; i < nk; i += 256) {
        const unsigned long long v = __ldg(src + i);
        key[i] = v;
        if (v) lo = min(lo, v);
        hi = max(hi, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (lane == 0) {
        ends[warp] = lo;
        ends[8 + warp] = hi;
    }
    __syncthreads();
    for (int w = 0; w < 8; ++w) {
        lo = min(lo, ends[w]);
        hi = max(hi, ends[8 + w]);
    }
    auto block_sum = [&](int n) {
        n = __reduce_add_sync(0xffffffffu, n);
        __syncthreads();
        if (lane == 0) sums[warp] = n;
        __syncthreads();
        int s = 0;
        for (int w = 0; w < 8; ++w) s += sums[w];
        return s;
    };
    auto count = [&](unsigned long long at) {
        int n = 0;
        for (int i = tid; i < nk; i += 256) n += key[i] >= at;
        return block_sum(n);
    };
    const int allowed = count(1);
    const int take = min(topk, allowed);
    unsigned long long at = lo;
    int n_at = allowed;
    while (n_at != take && lo < hi) {
        const unsigned long long mid = lo + ((hi - lo) >> 1) + 1;
        const int n = count(mid);
        if (n >= take) {
            lo = mid;
            at = mid;
            n_at = n;
        } else {
            hi = mid - 1;
        }
    }
    int ties = take;
    if (n_at != take) ties = take - (at == ~0ull ? 0 : count(at + 1));
    int written = 0;
    int* dst = blocks + row * topk;
    for (int i0 = 0; i0 < nk; i0 += 256) {
        const int i = i0 + tid;
        const unsigned long long v = i < nk ? key[i] : 0ull;
        const bool eq = v == at && v != 0;
        const unsigned equal = __ballot_sync(0xffffffffu, eq);
        __syncthreads();
        if (lane == 0) sums[warp] = __popc(equal);
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < 8; ++w) {
            before += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        const bool mine = take > 0 && (v > at || (eq && before + __popc(equal & ((1u << lane) - 1)) < ties));
        const unsigned pick = __ballot_sync(0xffffffffu, mine);
        __syncthreads();
        if (lane == 0) sums[warp] = __popc(pick);
        __syncthreads();
        int to = written;
        for (int w = 0; w < 8; ++w) {
            to += w < warp ? sums[w] : 0;
            written += sums[w];
        }
        if (mine) dst[to + __popc(pick & ((1u << lane) - 1))] = i;
        ties -= min(ties, all);
    }
    for (int i = written + tid; i < topk; i += 256) dst[i] = -1;
    if (tid == 0) counts[row] = take;
}

constexpr int SCORE64_SMEM = (128 * SCORE_Q + SCORE_K * K_PITCH) * 8;
constexpr int TOPK64_SMEM = 225 * 1024;

template <int NPL = 4>
void topk(const TopkParams& p, long long bh, cudaStream_t stream) {
    if constexpr (NPL < MAX_FAST / 32)
        if (p.nk > 32 * NPL) return topk<NPL + (NPL < 32 ? 4 : 16)>(p, bh, stream);
    block_topk_kernel<NPL><<<dim3((p.nq + 3) / 4, (unsigned)bh), 128, 0, stream>>>(p);
}

}  // namespace

int block_select_max_blocks() { return TOPK64_SMEM / 8; }

long long block_select_workspace(int B, int heads, const BlockGrid& g) {
    const long long nq = g.q_blocks(), nk = g.k_blocks();
    const long long means = (nq + nk) * 128 * 8 + nq * nk * 8;
    const long long pitch = (nk + 3) / 4 * 4;
    const long long fast = nk <= MAX_FAST ? (nq + nk) * 128 * 2 + (nq + pitch + nq * pitch) * 4 : 0;
    return (long long)B * heads * (means + fast) + 64;
}

cudaError_t init_block_select_attributes() {
    cudaError_t e = cudaFuncSetAttribute(block_score64_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SCORE64_SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(block_topk64_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TOPK64_SMEM);
    return e;
}

cudaError_t launch_block_select(const void* q, long long ldq, const void* k, long long ldk, int B, int heads,
                                const BlockGrid& g, const uint8_t* mask, int topk_, int* blocks, int* counts, void* ws,
                                const LaunchCtx& ctx) {
    const int nq = g.q_blocks(), nk = g.k_blocks();
    const long long bh = (long long)B * heads, rows = bh * nq;
    const bool fast = nk <= MAX_FAST;
    // workspace: 8-byte values first, then the 16-byte aligned fp16 units and fp32 rows
    double* qm = reinterpret_cast<double*>(ws);
    double* km = qm + bh * nq * 128;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(km + bh * nk * 128);  // [rows, nk]
    MeanOut oq{qm, nullptr, nullptr, 0}, ok{km, nullptr, nullptr, 0};
    float* scores = nullptr;
    const int pitch = (nk + 3) / 4 * 4;
    if (fast) {
        uintptr_t at = (reinterpret_cast<uintptr_t>(keys + rows * nk) + 15) & ~uintptr_t(15);
        oq.unit = reinterpret_cast<__half*>(at);
        ok.unit = oq.unit + bh * nq * 128;
        scores = reinterpret_cast<float*>(ok.unit + bh * nk * 128);
        ok.norm = scores + rows * pitch;
        ok.norm_pitch = pitch;
        oq.norm = ok.norm + bh * pitch;
        oq.norm_pitch = nq;
    }
    const int vecs = heads * 16;
    auto mean = [&](auto kernel, int most, int groups) {
        // the column slice that leaves the fewest threads idle, the widest of those (640 vectors:
        // 160 threads 249 us, 256 with a sixth of them idle 290)
        int threads = 32, idle = INT_MAX;
        for (int n = 32; n <= most; n += 32) {
            const int rest = (vecs + n - 1) / n * n - vecs;
            if (rest <= idle) {
                idle = rest;
                threads = n;
            }
        }
        kernel<<<dim3(nq + nk, (vecs + threads - 1) / threads, B), dim3(threads, groups), 0, ctx.stream>>>(
            reinterpret_cast<const __nv_bfloat16*>(q), ldq, reinterpret_cast<const __nv_bfloat16*>(k), ldk, heads, g, oq, ok);
    };
    // under an SM's 1024 threads on each: four groups of threads per slice
    if ((long long)(nq + nk) * vecs * B < 148 * 1024) mean(block_mean_kernel<4>, 64, 4);
    else mean(block_mean_kernel<1>, 256, 1);
    if (fast) {
        block_score_kernel<<<dim3((nk + ST - 1) / ST, (nq + ST - 1) / ST, (unsigned)bh), 128, 0, ctx.stream>>>(
            oq.unit, ok.unit, ok.norm, nq, nk, pitch, scores);
        const TopkParams p{scores, qm, km, oq.norm, ok.norm, mask, keys, nq, nk, pitch, topk_, blocks, counts};
        topk(p, bh, ctx.stream);
    } else {
        block_score64_kernel<<<dim3((nk + SCORE_K - 1) / SCORE_K, (nq + SCORE_Q - 1) / SCORE_Q, (unsigned)bh), 128,
                               SCORE64_SMEM, ctx.stream>>>(qm, km, mask, nq, nk, keys);
        block_topk64_kernel<<<(unsigned)rows, 256, nk * 8, ctx.stream>>>(keys, nk, topk_, blocks, counts);
    }
    if (ctx.launches) *ctx.launches += 3;
    return cudaGetLastError();
}

}  // namespace wan
