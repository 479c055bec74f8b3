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
//   block_mean_kernel   one pass over q and k: fp64 means, their bf16 hi + lo
//                       parts and their norms;
//   block_score_kernel  scores from three bf16 products (hi hi + hi lo + lo hi) on
//                       the tensor cores, fp32 sums; every score is within
//                       SCORE_ERROR |q| |k| of its 64-bit value;
//   block_topk_kernel   the topk-th best of a row by bisection; only blocks whose
//                       score lies within the error of it are scored again, in
//                       fp64, and ranked by that (none or a few per row).
// Longer rows: block_score64_kernel and block_topk64_kernel, all in fp64.
#include "common.cuh"
#include "kernels.h"

namespace wan {

namespace {

constexpr int SCORE_Q = 32, SCORE_K = 64;  // fp64 score kernel: query x key blocks per CTA
constexpr int K_PITCH = 129;               // doubles per staged mean (odd: column reads hit all banks)
constexpr int MAX_FAST = 2048;             // key blocks of the two-stage path
// Bound of a tensor-core score's error over |q| |k|: a bf16 rounding is off by
// 2^-8, so lo misses 2^-16 of each factor and lo lo is another 2^-16 (4.6e-5 in
// all); 384 fp32 additions, truncated, add at most 384 * 2^-23 (4.6e-5).
constexpr float SCORE_ERROR = 1.220703125e-4f;  // 2^-13
constexpr float SCORE_TINY = 1e-34f;            // below it products lose bits to underflow

// Means of the blocks of q (first g.q_blocks() CTAs) and k, per head: fp64, bf16
// hi | lo parts [256] and norm.  One CTA per block and 256-thread column slice,
// eight columns per thread; four tokens are added in fp32 before they join the
// fp64 sum: bf16 has 8 significant bits, so a sum of four of them is exact in
// fp32's 24 unless their exponents lie 14 apart.
struct MeanOut {
    double* mean;           // [B, heads, blocks, 128]
    __nv_bfloat16* parts;   // [B, heads, blocks, 256], null: not wanted
    float* norm;            // [B, heads, blocks]
};
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
    for (int t = threadIdx.x; t < n; t += blockDim.x)
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
        float s[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 p = unpack_bf16(w[c]);
                s[2 * c] = u ? s[2 * c] + p.x : p.x;
                s[2 * c + 1] = u ? s[2 * c + 1] + p.y : p.y;
            }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] += (double)s[c];
    };
    int t = 0;
    for (; t + 8 <= n; t += 8) {
        uint4 v[2][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u >> 2][u & 3] = __ldg(reinterpret_cast<const uint4*>(base + (long long)tokens[t + u] * ld));
        add(v[0]);
        add(v[1]);
    }
    for (; t < n; t += 4) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] = t + u < n ? __ldg(reinterpret_cast<const uint4*>(base + (long long)tokens[t + u] * ld)) : make_uint4(0, 0, 0, 0);
        add(v);
    }
    const MeanOut& o = keys ? ok : oq;
    const long long at = ((long long)b * heads + (mine ? col / 128 : 0)) * (nF * nH * nW) + blk;
    const double count = (double)n;
    float hi[8], lo[8], ss = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        acc[c] /= count;
        hi[c] = __bfloat162float(__float2bfloat16_rn((float)acc[c]));
        lo[c] = (float)(acc[c] - (double)hi[c]);
        ss += (float)acc[c] * (float)acc[c];
    }
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
    if (!mine) return;
    double* dst = o.mean + at * 128 + col % 128;
#pragma unroll
    for (int c = 0; c < 8; c += 2) *reinterpret_cast<double2*>(dst + c) = make_double2(acc[c], acc[c + 1]);
    if (!o.parts) return;
    __nv_bfloat16* parts = o.parts + at * 256 + col % 128;
    *reinterpret_cast<uint4*>(parts) =
        make_uint4(pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3]), pack_bf16(hi[4], hi[5]), pack_bf16(hi[6], hi[7]));
    *reinterpret_cast<uint4*>(parts + 128) =
        make_uint4(pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]), pack_bf16(lo[4], lo[5]), pack_bf16(lo[6], lo[7]));
    if ((threadIdx.x & 15) == 0) o.norm[at] = sqrtf(ss) * 1.0001f;
}

// ---------------------------------------------------------------- two-stage path
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// scores[bh][i][j] = hi hi + hi lo + lo hi of the means' parts.  64 x 64 scores per
// CTA, four warps of 32 x 32; both operands whole (K = 128) in shared memory, 512
// bytes a row, 16-byte pieces swizzled by the row.  mma.sync and not tcgen05: the
// products are a few microseconds of work in tiles too small to fill a 128-row
// accumulator per head.
constexpr int ST = 64;
__global__ void __launch_bounds__(128) block_score_kernel(const __nv_bfloat16* __restrict__ qp, const __nv_bfloat16* __restrict__ kp,
                                                          int nq, int nk, float* __restrict__ scores) {
    extern __shared__ uint4 tile[];  // [2][ST][32]
    const int q0 = blockIdx.y * ST, k0 = blockIdx.x * ST;
    const long long bh = blockIdx.z;
    for (int i = threadIdx.x; i < 2 * ST * 32; i += 128) {
        const int which = i / (ST * 32), r = i / 32 % ST, c = i % 32;
        const int at = (which ? k0 : q0) + r, n = which ? nk : nq;
        const __nv_bfloat16* src = (which ? kp : qp) + (bh * n + at) * 256 + c * 8;
        tile[(which * ST + r) * 32 + (c ^ (r & 7))] = at < n ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m0 = (warp >> 1) * 32, n0 = (warp & 1) * 32;
    const uint32_t sq = smem_u32(tile), sk = sq + ST * 512;
    float acc[2][4][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][j][c] = 0.f;
    // 8 x 8 matrices of a x4 load: rows lane & 7 (+ 8), 16-byte piece 2 kk (+ 1); part: 0 hi, 16 lo
    auto load_a = [&](uint32_t (&r)[4], int row, int kk, int part) {
        const int at = row + (lane & 15), c = part + 2 * kk + (lane >> 4);
        ldmatrix4(r, sq + at * 512 + ((c ^ (at & 7)) << 4));
    };
    auto load_b = [&](uint32_t (&r)[4], int row, int kk, int part) {  // two n8 tiles
        const int at = row + (lane & 7) + ((lane >> 4) << 3), c = part + 2 * kk + ((lane >> 3) & 1);
        ldmatrix4(r, sk + at * 512 + ((c ^ (at & 7)) << 4));
    };
#pragma unroll 2
    for (int kk = 0; kk < 8; ++kk) {
        uint32_t ah[2][4], al[2][4], bh4[2][4], bl4[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            load_a(ah[i], m0 + 16 * i, kk, 0);
            load_a(al[i], m0 + 16 * i, kk, 16);
            load_b(bh4[i], n0 + 16 * i, kk, 0);
            load_b(bl4[i], n0 + 16 * i, kk, 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t h0 = bh4[j >> 1][(j & 1) * 2], h1 = bh4[j >> 1][(j & 1) * 2 + 1];
                mma_16816(acc[i][j], ah[i], bl4[j >> 1][(j & 1) * 2], bl4[j >> 1][(j & 1) * 2 + 1]);
                mma_16816(acc[i][j], al[i], h0, h1);
                mma_16816(acc[i][j], ah[i], h0, h1);
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = q0 + m0 + 16 * i + half * 8 + (lane >> 2);
            if (row >= nq) continue;
            float* dst = scores + (bh * nq + row) * nk;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = k0 + n0 + 8 * j + (lane & 3) * 2;
                if (col < nk) dst[col] = acc[i][j][half * 2];
                if (col + 1 < nk) dst[col + 1] = acc[i][j][half * 2 + 1];
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

// The topk best blocks of a row: one warp per row, NPL scores per lane in
// registers (nk <= 32 NPL).  Bisection between the row's smallest and largest key
// ends as soon as a threshold leaves exactly topk of them (a dozen steps).  Blocks
// whose score lies within twice the error bound of the topk-th are ranked by their
// fp64 scores, equal ones to the lower block.
struct TopkParams {
    const float* scores;            // [B heads nq, nk]
    const double *qm, *km;          // means
    const float *qn, *kn;           // their norms
    const uint8_t* mask;            // [nq, nk] or null
    unsigned long long* exact;      // [rows, nk]: used by rows with many close scores only
    int nq, nk, topk;
    long long rows;
    int *blocks, *counts;
};
template <int NPL>
__global__ void __launch_bounds__(128) block_topk_kernel(const __grid_constant__ TopkParams p) {
    const int lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const int nk = p.nk;
    const long long bh = row / p.nq;
    const float* src = p.scores + row * nk;
    const uint8_t* mrow = p.mask ? p.mask + (row - bh * p.nq) * nk : nullptr;
    const float* kn = p.kn + bh * nk;
    uint32_t key[NPL];
    uint32_t lo = ~0u, hi = 0;
    float far = 0.f;  // largest key norm, NaN if one is
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int j = i * 32 + lane;
        key[i] = 0;
        if (j < nk) {
            key[i] = score_key32(__ldg(src + j));
            if (mrow) {
                const uint8_t m = __ldg(mrow + j);
                key[i] = m == 0 ? 0u : m == 1 ? key[i] : ~0u;
            }
            const float x = __ldg(kn + j);
            far = x > far || !(x == x) ? x : far;
        }
        if (key[i] != 0) lo = min(lo, key[i]);
        hi = max(hi, key[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    auto count = [&](uint32_t at) {  // keys >= at
        int n = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) n += key[i] >= at;
        return (int)__reduce_add_sync(0xffffffffu, n);
    };
    const int allowed = count(1);
    const int take = min(p.topk, allowed);
    // count(at) >= take, and == take unless equal keys lie at the border
    uint32_t at = lo;
    int n_at = allowed;
    while (n_at != take && lo < hi) {
        const uint32_t mid = lo + ((hi - lo) >> 1) + 1;
        const int n = count(mid);
        if (n >= take) {
            lo = mid;
            at = mid;
            n_at = n;
        } else {
            hi = mid - 1;
        }
    }
    int* dst = p.blocks + row * p.topk;
    int written = 0;
    auto put = [&](int i, bool pick) {
        const unsigned picks = __ballot_sync(0xffffffffu, pick);
        if (pick) dst[written + __popc(picks & below)] = i * 32 + lane;
        written += __popc(picks);
    };
    // the topk-th score and the best one that is left out
    uint32_t vk = ~0u, vn = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        if (key[i] >= at) vk = min(vk, key[i]);
        else vn = max(vn, key[i]);
    }
    vk = __reduce_min_sync(0xffffffffu, vk);
    vn = __reduce_max_sync(0xffffffffu, vn);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, far, o);
        far = x > far || !(x == x) ? x : far;
    }
    const float reach = 2.0f * (SCORE_ERROR * p.qn[row] * far + SCORE_TINY);
    const float border = key32_score(vk);
    if (take == 0 || vk == ~0u) {
        // nothing, or blocks asked for alone: the lowest of them
        int left = take;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const unsigned all = __ballot_sync(0xffffffffu, key[i] == ~0u);
            put(i, key[i] == ~0u && __popc(all & below) < left);
            left -= min(left, __popc(all));
        }
    } else if (n_at == take && (vn == 0 || border - key32_score(vn) > reach)) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) put(i, key[i] >= at);
    } else {
        // close: 1 (ranked again); 2: taken for sure (also when reach is not a number: all are close)
        auto kind = [&](uint32_t k) -> int {
            if (k == 0) return 0;
            if (k == ~0u) return 2;
            const float s = key32_score(k);
            return s > border + reach ? 2 : s < border - reach ? 0 : 1;
        };
        int close = 0, sure = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int x = kind(key[i]);
            close += x == 1;
            sure += x == 2;
        }
        close = __reduce_add_sync(0xffffffffu, close);
        sure = __reduce_add_sync(0xffffffffu, sure);
        const double* qd = p.qm + row * 128 + lane * 4;
        const double qx[4] = {qd[0], qd[1], qd[2], qd[3]};
        auto exact_key = [&](int j) {  // all lanes: 64-bit key of block j
            const double2* kd = reinterpret_cast<const double2*>(p.km + (bh * nk + j) * 128 + lane * 4);
            const double2 k0 = __ldg(kd), k1 = __ldg(kd + 1);
            double s = fma(qx[3], k1.y, fma(qx[2], k1.x, fma(qx[1], k0.y, qx[0] * k0.x)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            return score_key(s);
        };
        if (close <= 32) {
            // lane n holds the n-th close block
            unsigned long long mine = 0;
            int n = 0;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                unsigned here = __ballot_sync(0xffffffffu, kind(key[i]) == 1);
                while (here) {
                    const int l = __ffs(here) - 1;
                    here &= here - 1;
                    const unsigned long long k = exact_key(i * 32 + l);
                    if (lane == n) mine = k;
                    ++n;
                }
            }
            int better = 0;
            for (int l = 0; l < close; ++l) {
                const unsigned long long k = __shfl_sync(0xffffffffu, mine, l);
                better += k > mine || (k == mine && l < lane);
            }
            const unsigned chosen = __ballot_sync(0xffffffffu, lane < close && better < take - sure);
            int seen = 0;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int x = kind(key[i]);
                const unsigned here = __ballot_sync(0xffffffffu, x == 1);
                put(i, x == 2 || (x == 1 && (chosen >> ((seen + __popc(here & below)) & 31) & 1)));
                seen += __popc(here);
            }
        } else {
            // many close scores (equal blocks, infinities): all fp64 keys through memory
            unsigned long long* ek = p.exact + row * nk;
            unsigned long long lo64 = ~0ull, hi64 = 0;
#pragma unroll 1
            for (int i0 = 0; i0 < nk; i0 += 32) {
                const int j = i0 + lane;
                uint32_t k32 = 0;
#pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if (i * 32 == i0) k32 = key[i];
                const int x = kind(k32);
                unsigned long long k = x == 2 ? ~0ull : 0ull;
                unsigned here = __ballot_sync(0xffffffffu, x == 1);
                while (here) {
                    const int l = __ffs(here) - 1;
                    here &= here - 1;
                    const unsigned long long e = exact_key(i0 + l);
                    if (lane == l) k = e;
                }
                if (j < nk) ek[j] = k;
                if (k) lo64 = min(lo64, k);
                hi64 = max(hi64, k);
            }
            __syncwarp();
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                lo64 = min(lo64, __shfl_xor_sync(0xffffffffu, lo64, o));
                hi64 = max(hi64, __shfl_xor_sync(0xffffffffu, hi64, o));
            }
            auto count64 = [&](unsigned long long v) {
                int n = 0;
                for (int j = lane; j < nk; j += 32) n += ek[j] >= v;
                return (int)__reduce_add_sync(0xffffffffu, n);
            };
            unsigned long long at64 = lo64;
            int n64 = close + sure;
            while (n64 != take && lo64 < hi64) {
                const unsigned long long mid = lo64 + ((hi64 - lo64) >> 1) + 1;
                const int n = count64(mid);
                if (n >= take) {
                    lo64 = mid;
                    at64 = mid;
                    n64 = n;
                } else {
                    hi64 = mid - 1;
                }
            }
            int ties = n64 == take ? take : take - count64(at64 + 1);  // at64 < ~0: fewer than take are sure
            for (int i0 = 0; i0 < nk; i0 += 32) {
                const int j = i0 + lane;
                const unsigned long long k = j < nk ? ek[j] : 0ull;
                const unsigned equal = __ballot_sync(0xffffffffu, k == at64 && k != 0);
                put(i0 / 32, k > at64 || (k == at64 && k != 0 && __popc(equal & below) < ties));
                ties -= min(ties, __popc(equal));
            }
        }
    }
    for (int i = written + lane; i < p.topk; i += 32) dst[i] = -1;
    if (lane == 0) p.counts[row] = take;
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

constexpr int SCORE_SMEM = 2 * ST * 512;
constexpr int SCORE64_SMEM = (128 * SCORE_Q + SCORE_K * K_PITCH) * 8;
constexpr int TOPK64_SMEM = 225 * 1024;

template <int NPL>
void topk(const TopkParams& p, cudaStream_t stream) {
    block_topk_kernel<NPL><<<(unsigned)((p.rows + 3) / 4), 128, 0, stream>>>(p);
}

}  // namespace

int block_select_max_blocks() { return TOPK64_SMEM / 8; }

long long block_select_workspace(int B, int heads, const BlockGrid& g) {
    const long long nq = g.q_blocks(), nk = g.k_blocks();
    const long long each = nk <= MAX_FAST ? (nq + nk) * (128 * 8 + 256 * 2 + 4) + nq * nk * 12 : (nq + nk) * 128 * 8 + nq * nk * 8;
    return (long long)B * heads * each + 64;
}

cudaError_t init_block_select_attributes() {
    cudaError_t e = cudaFuncSetAttribute(block_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SCORE_SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(block_score64_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SCORE64_SMEM);
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
    // workspace: 8-byte values first, then 16-byte aligned parts, then fp32
    double* qm = reinterpret_cast<double*>(ws);
    double* km = qm + bh * nq * 128;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(km + bh * nk * 128);  // [rows, nk]
    MeanOut oq{qm, nullptr, nullptr}, ok{km, nullptr, nullptr};
    float* scores = nullptr;
    if (fast) {
        uintptr_t at = (reinterpret_cast<uintptr_t>(keys + rows * nk) + 15) & ~uintptr_t(15);
        oq.parts = reinterpret_cast<__nv_bfloat16*>(at);
        ok.parts = oq.parts + bh * nq * 256;
        oq.norm = reinterpret_cast<float*>(ok.parts + bh * nk * 256);
        ok.norm = oq.norm + bh * nq;
        scores = ok.norm + bh * nk;
    }
    const int vecs = heads * 16;
    const int threads = vecs < 256 ? (vecs + 31) / 32 * 32 : 256;
    const int slices = (vecs + threads - 1) / threads;
    block_mean_kernel<<<dim3(nq + nk, slices, B), threads, 0, ctx.stream>>>(
        reinterpret_cast<const __nv_bfloat16*>(q), ldq, reinterpret_cast<const __nv_bfloat16*>(k), ldk, heads, g, oq, ok);
    if (fast) {
        block_score_kernel<<<dim3((nk + ST - 1) / ST, (nq + ST - 1) / ST, (unsigned)bh), 128, SCORE_SMEM, ctx.stream>>>(
            oq.parts, ok.parts, nq, nk, scores);
        const TopkParams p{scores, qm, km, oq.norm, ok.norm, mask, keys, nq, nk, topk_, rows, blocks, counts};
        const int per_lane = (nk + 31) / 32;
        if (per_lane <= 4) topk<4>(p, ctx.stream);
        else if (per_lane <= 12) topk<12>(p, ctx.stream);
        else if (per_lane <= 20) topk<20>(p, ctx.stream);
        else if (per_lane <= 32) topk<32>(p, ctx.stream);
        else topk<64>(p, ctx.stream);
    } else {
        block_score64_kernel<<<dim3((nk + SCORE_K - 1) / SCORE_K, (nq + SCORE_Q - 1) / SCORE_Q, (unsigned)bh), 128,
                               SCORE64_SMEM, ctx.stream>>>(qm, km, mask, nq, nk, keys);
        block_topk64_kernel<<<(unsigned)rows, 256, nk * 8, ctx.stream>>>(keys, nk, topk_, blocks, counts);
    }
    if (ctx.launches) *ctx.launches += 3;
    return cudaGetLastError();
}

}  // namespace wan
