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
//   block_topk_kernel   the topk-th best of a row by bisection; only blocks that
//                       the error lets lie on either side of the border (seven or
//                       so of several hundred) are scored again, in fp64, and
//                       ranked by that.
// (With hi + lo parts and three products fewer are scored again, but the products
// and their operands cost more than that saves: 30 against 12 us of the pair's.)
// Longer rows: block_score64_kernel and block_topk64_kernel, all in fp64.
#include <cuda_fp16.h>

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
// column slice, eight columns per thread, four tokens loaded while the four before
// are added; where there are few CTAs (a small grid) RG = 4 groups of threads take
// every fourth eight tokens each: a block is a chain of loads (14.5 -> 7.6 us at 15
// blocks).  Every token is added in fp64: it must not matter what stands beside a
// small one.  (Sums of four tokens in fp32 first, which lose a value 2^17 times
// smaller than its neighbour, took 70 us where this takes 72; the same with the
// rounding errors kept beside them 133.)  The conversions to fp64, at 16 a clock and
// SM, are two thirds busy then; the loads are what bounds it.
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
            v[u] = t + u < n ? __ldg(reinterpret_cast<const uint4*>(base + (long long)tokens[t + u] * ld)) : make_uint4(0, 0, 0, 0);
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
    const double count = (double)n;
    double ss = 0.0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        acc[c] /= count;
        ss += acc[c] * acc[c];
    }
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
// rows `pitch` apart.  64 x 64 scores per CTA, four warps of 32 x 32; both operands
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
        if (col >= nk) continue;
        const float s0 = __ldg(kn + bh * pitch + col), s1 = col + 1 < nk ? __ldg(kn + bh * pitch + col + 1) : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = q0 + m0 + 16 * i + half * 8 + (lane >> 2);
                if (row < nq)
                    *reinterpret_cast<float2*>(scores + (bh * nq + row) * pitch + col) =
                        make_float2(acc[i][j][half * 2] * s0, acc[i][j][half * 2 + 1] * s1);
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

// The topk best blocks of a row: one warp per row, a lane holding the keys of NPL
// consecutive blocks in registers (nk <= 32 NPL).  A threshold that leaves topk
// keys is found by interpolation and bisection in turn (half a dozen counts).
// With a_j the fp32 score of block j and d_j the bound of its error, the topk-th
// best 64-bit score is at least L = min (a_j - d_j) over the topk best a_j and at
// most U = max (a_j + d_j) over the topk-th and all others: blocks with a_j - d_j >
// U are taken, those with a_j + d_j < L are not, and the close ones in between are
// ranked by their fp64 scores, equal ones to the lower block.
struct TopkParams {
    const float* scores;            // [B heads nq, pitch]
    const double *qm, *km;          // means
    const float *qn, *kn;           // their norms: [B heads, nq], [B heads, pitch]
    const uint8_t* mask;            // [nq, nk] or null
    unsigned long long* exact;      // [rows, nk]: used by rows with many close scores only
    int nq, nk, pitch, topk;
    int *blocks, *counts;
};
template <int NPL>
__global__ void __launch_bounds__(128, NPL <= 24 ? 8 : 1) block_topk_kernel(const __grid_constant__ TopkParams p) {
    using Bits = typename std::conditional<(NPL > 32), unsigned long long, uint32_t>::type;
    // rows come in coalesced and are read back a lane's consecutive blocks at a time
    __shared__ int again[4][32];
    __shared__ float4 norms[NPL * 8], stage[4][NPL * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nk = p.nk, j0 = lane * NPL;  // the lane's first block
    const long long bh = blockIdx.y;
    const int i_q = blockIdx.x * 4 + warp;
    const long long row = bh * p.nq + i_q;
    bool number = true;  // every norm of the head is one
    for (int i = threadIdx.x; i < NPL * 8; i += 128) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < p.pitch / 4) {
            v = __ldg(reinterpret_cast<const float4*>(p.kn + bh * p.pitch) + i);
            const int rest = nk - 4 * i;
            number = number && v.x < INFINITY && (rest < 2 || v.y < INFINITY) && (rest < 3 || v.z < INFINITY) &&
                     (rest < 4 || v.w < INFINITY);
        }
        norms[i] = v;
    }
    if (i_q < p.nq) {
        const float4* src = reinterpret_cast<const float4*>(p.scores + row * p.pitch);
#pragma unroll
        for (int i = 0; i < NPL / 4; ++i)
            if (i * 32 + lane < p.pitch / 4) stage[warp][i * 32 + lane] = __ldg(src + i * 32 + lane);
    }
    number = __syncthreads_and(number);
    if (i_q >= p.nq) return;
    // scores of the allowed blocks; NaN, which no comparison holds for, where there is none or
    // it is not the score that decides: `extra` are the blocks asked for
    float f[NPL];
    Bits extra = 0;
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
        const float4 v = stage[warp][(j0 + i) / 4];
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) f[i + c] = j0 + i + c < nk ? (x[c] == x[c] ? x[c] : -INFINITY) : NAN;
    }
    if (p.mask) {
        const uint8_t* mrow = p.mask + (long long)i_q * nk + j0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const uint8_t m = j0 + i < nk ? __ldg(mrow + i) : 0;
            f[i] = m == 1 ? f[i] : NAN;
            extra |= (Bits)(m > 1) << i;
        }
    }
    auto bits_of = [](Bits x) { return NPL > 32 ? __popcll(x) : __popc((uint32_t)x); };
    auto count = [&](float at) {  // scores >= at
        int n = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) n += f[i] >= at;
        return (int)__reduce_add_sync(0xffffffffu, n);
    };
    const int always = p.mask ? __reduce_add_sync(0xffffffffu, bits_of(extra)) : 0;
    const int scored = p.mask ? count(-INFINITY) : nk;
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
        Bits all = extra;
#pragma unroll
        for (int i = 0; i < NPL; ++i) all |= (Bits)(f[i] == f[i]) << i;
        put(all);
        return;
    }
    // at: a score that `want` scores reach, and no more unless equal ones lie at the border.  The
    // first place is where normally distributed scores would have it, the next ones are taken by
    // the counts, every third half way (five counts for a normal row, ten without the first
    // guess); where that does not settle it (infinities, scores of many magnitudes) half way
    // between the scores' bit patterns.
    float lo = INFINITY, hi = -INFINITY, sum = 0.f, sum2 = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        lo = fminf(lo, f[i]);
        hi = fmaxf(hi, f[i]);
        const float x = f[i] == f[i] ? f[i] : 0.f;
        sum += x;
        sum2 = fmaf(x, x, sum2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum2 += __shfl_xor_sync(0xffffffffu, sum2, o);
    }
    const float mean = sum / scored, spread = sqrtf(fmaxf(sum2 / scored - mean * mean, 0.f));
    const float guess = mean + spread * 0.4073f * log2f((float)(scored - want) / (float)want);  // ln 2 / 1.702
    float at = lo;
    int n_at = scored, n_hi = 0;  // n_hi: scores >= the last place that was too high
    for (int step = 0; n_at != want && lo < hi; ++step) {
        const float part = step % 3 == 0 ? 0.5f : fminf(fmaxf((float)(n_at - want) / (float)(n_at - n_hi), 0.05f), 0.95f);
        float mid = step == 0 && guess > lo && guess < hi ? guess : lo + part * (hi - lo);
        if (step >= 24 || !(mid > lo && mid <= hi)) {
            const uint32_t a = score_key32(lo), b = score_key32(hi);
            mid = key32_score(a + ((b - a) >> 1) + 1);
        }
        const int n = count(mid);
        if (n >= want) {
            lo = at = mid;
            n_at = n;
        } else {
            hi = key32_score(score_key32(mid) - 1);  // the next lower float
            n_hi = n;
        }
    }
    // L, U and the close ones
    const float4* kn = norms + j0 / 4;
    float L = INFINITY, U = -INFINITY, vk = INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) vk = fminf(vk, f[i] >= at ? f[i] : INFINITY);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) vk = fminf(vk, __shfl_xor_sync(0xffffffffu, vk, o));
    float d[4];
    auto bounds = [&](int i) {  // of four blocks
        const float4 v = kn[i / 4];
        d[0] = fmaf(SCORE_ERROR, v.x, SCORE_TINY);
        d[1] = fmaf(SCORE_ERROR, v.y, SCORE_TINY);
        d[2] = fmaf(SCORE_ERROR, v.z, SCORE_TINY);
        d[3] = fmaf(SCORE_ERROR, v.w, SCORE_TINY);
    };
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        if (i % 4 == 0) bounds(i);
        L = fminf(L, f[i] >= at ? f[i] - d[i % 4] : INFINITY);
        U = fmaxf(U, f[i] <= vk ? f[i] + d[i % 4] : -INFINITY);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        L = fminf(L, __shfl_xor_sync(0xffffffffu, L, o));
        U = fmaxf(U, __shfl_xor_sync(0xffffffffu, U, o));
    }
    Bits sure = extra, close = 0;
    if (number && p.qn[row] < INFINITY) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (i % 4 == 0) bounds(i);
            const bool in = f[i] - d[i % 4] > U;
            sure |= (Bits)in << i;
            close |= (Bits)(!in && f[i] + d[i % 4] >= L) << i;
        }
    } else {  // a mean is not finite: all are close
#pragma unroll
        for (int i = 0; i < NPL; ++i) close |= (Bits)(f[i] == f[i]) << i;
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
        // lane n ranks the n-th close block among all of them
        const int first = before(close);
        Bits rest = close;
        for (int n = first; rest; ++n) {
            const Bits low = rest & (~rest + 1);
            again[warp][n] = j0 + bits_of(low - 1);
            rest ^= low;
        }
        __syncwarp();
        unsigned long long k = 0;
#pragma unroll 1
        for (int c = 0; c < n_close; c += 4) {
            const unsigned long long e = exact_key(again[warp][min(c + (lane >> 3), n_close - 1)]);
            const unsigned long long got = __shfl_sync(0xffffffffu, e, (lane & 3) * 8);
            if (lane >= c && lane < c + 4) k = got;  // c is a multiple of 4: lane & 3 == lane - c
        }
        int better = 0;
        for (int l = 0; l < n_close; ++l) {
            const unsigned long long other = __shfl_sync(0xffffffffu, k, l);
            better += other > k || (other == k && l < lane);
        }
        const unsigned chosen = __ballot_sync(0xffffffffu, lane < n_close && better < need);
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

template <int NPL>
void topk(const TopkParams& p, long long bh, cudaStream_t stream) {
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
        const int threads = vecs < most ? (vecs + 31) / 32 * 32 : most;
        kernel<<<dim3(nq + nk, (vecs + threads - 1) / threads, B), dim3(threads, groups), 0, ctx.stream>>>(
            reinterpret_cast<const __nv_bfloat16*>(q), ldq, reinterpret_cast<const __nv_bfloat16*>(k), ldk, heads, g, oq, ok);
    };
    if ((long long)(nq + nk) * vecs * B < 148 * 1024) mean(block_mean_kernel<4>, 64, 4);
    else mean(block_mean_kernel<1>, 256, 1);
    if (fast) {
        block_score_kernel<<<dim3((nk + ST - 1) / ST, (nq + ST - 1) / ST, (unsigned)bh), 128, 0, ctx.stream>>>(
            oq.unit, ok.unit, ok.norm, nq, nk, pitch, scores);
        const TopkParams p{scores, qm, km, oq.norm, ok.norm, mask, keys, nq, nk, pitch, topk_, blocks, counts};
        const int per_lane = (nk + 31) / 32;
        if (per_lane <= 4) topk<4>(p, bh, ctx.stream);
        else if (per_lane <= 12) topk<12>(p, bh, ctx.stream);
        else if (per_lane <= 20) topk<20>(p, bh, ctx.stream);
        else if (per_lane <= 24) topk<24>(p, bh, ctx.stream);
        else if (per_lane <= 32) topk<32>(p, bh, ctx.stream);
        else topk<64>(p, bh, ctx.stream);
    } else {
        block_score64_kernel<<<dim3((nk + SCORE_K - 1) / SCORE_K, (nq + SCORE_Q - 1) / SCORE_Q, (unsigned)bh), 128,
                               SCORE64_SMEM, ctx.stream>>>(qm, km, mask, nq, nk, keys);
        block_topk64_kernel<<<(unsigned)rows, 256, nk * 8, ctx.stream>>>(keys, nk, topk_, blocks, counts);
    }
    if (ctx.launches) *ctx.launches += 3;
    return cudaGetLastError();
}

}  // namespace wan
