// Choice of key blocks for block-sparse attention: the score of query block i
// and key block j of one head is the dot product of their mean query and mean
// key, and each query block keeps the topk best-scored key blocks.
//   block_mean_kernel   one pass over q and k: fp64 means of each block;
//   block_score_kernel  fp64 scores, stored as 64-bit keys in score order;
//   block_topk_*_kernel the topk largest keys of a row, written in block order.
// The choice is a comparison of scores that lie close together (a row of a few
// hundred scores has neighbours 1e-6 apart as a matter of course), so sums and
// products are held in 64 bits: a score depends on the inputs alone, not on the
// order of its additions.
#include "common.cuh"
#include "kernels.h"

namespace wan {

namespace {

constexpr int SCORE_Q = 32, SCORE_K = 64;  // query x key blocks per CTA of the score kernel
constexpr int K_PITCH = 129;               // doubles per staged mean (odd: column reads hit all banks)

// Means of the blocks of one tensor: out[b][h][block][128].  One CTA per block
// and 256-thread column slice, eight columns per thread; four tokens are added
// in fp32 before they join the fp64 sum: bf16 has 8 significant bits, so a sum
// of four of them is exact in fp32's 24 unless their exponents lie 14 apart.
__global__ void __launch_bounds__(256) block_mean_kernel(const __nv_bfloat16* __restrict__ x, long long ld, int heads,
                                                         int F, int H, int W, int bF, int bH, int bW,
                                                         double* __restrict__ out) {
    __shared__ int tokens[128];
    const int nH = (H + bH - 1) / bH, nW = (W + bW - 1) / bW, nF = (F + bF - 1) / bF;
    const int blk = blockIdx.x, b = blockIdx.z;
    const int f0 = blk / (nH * nW) * bF, i0 = blk / nW % nH * bH, j0 = blk % nW * bW;
    const int ef = min(bF, F - f0), ei = min(bH, H - i0), ej = min(bW, W - j0);
    const int n = ef * ei * ej;
    for (int t = threadIdx.x; t < n; t += blockDim.x)
        tokens[t] = ((f0 + t / (ej * ei)) * H + i0 + t / ej % ei) * W + j0 + t % ej;
    __syncthreads();
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    if (col >= heads * 128) return;
    const __nv_bfloat16* base = x + (long long)b * F * H * W * ld + col;
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
    double* dst = out + (((long long)b * heads + col / 128) * (nF * nH * nW) + blk) * 128 + col % 128;
    const double inv_n = (double)n;
#pragma unroll
    for (int c = 0; c < 8; c += 2) *reinterpret_cast<double2*>(dst + c) = make_double2(acc[c] / inv_n, acc[c + 1] / inv_n);
}

// A score as a 64-bit key in the same order: NaN ranks with -inf, keys of
// allowed blocks are above 0 and below ~0.
__device__ __forceinline__ unsigned long long score_key(double s) {
    if (!(s == s)) s = -INFINITY;
    if (s == 0.0) s = 0.0;  // -0 and 0 tie
    const unsigned long long u = (unsigned long long)__double_as_longlong(s);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// keys[bh][i][j] = key of (q mean i) . (k mean j); 0 where the mask forbids the
// block, ~0 where it asks for it.  Each thread 8 query x 2 key blocks.
__global__ void __launch_bounds__(128) block_score_kernel(const double* __restrict__ qm, const double* __restrict__ km,
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

// The topk largest keys of a row, by bisection between the row's smallest and
// largest key: most rows end as soon as a threshold leaves exactly topk keys
// (a dozen steps); equal keys at the border go to the lowest blocks.  One warp
// per row, NPL keys per lane in registers (nk <= 32 NPL).
template <int NPL>
__global__ void __launch_bounds__(128) block_topk_warp_kernel(const unsigned long long* __restrict__ keys, int nk,
                                                              int topk, long long rows, int* __restrict__ blocks,
                                                              int* __restrict__ counts) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const unsigned long long* src = keys + row * nk;
    unsigned long long key[NPL];
    unsigned long long lo = ~0ull, hi = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        key[i] = i * 32 + lane < nk ? __ldg(src + i * 32 + lane) : 0ull;
        if (key[i]) lo = min(lo, key[i]);
        hi = max(hi, key[i]);
    }
    auto count = [&](unsigned long long at) {  // keys >= at
        int n = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) n += key[i] >= at;
        return (int)__reduce_add_sync(0xffffffffu, n);
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const int allowed = count(1);
    const int take = min(topk, allowed);
    // invariant: count(lo) >= take and count(> hi) < take
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
    // keys above `at` are taken, of those equal to it the first `ties`
    int ties = take;
    if (n_at != take) ties = take - (at == ~0ull ? 0 : count(at + 1));
    int written = 0;
    int* dst = blocks + row * topk;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const unsigned equal = __ballot_sync(0xffffffffu, key[i] == at && key[i] != 0);
        const bool mine = key[i] > at || (key[i] == at && key[i] != 0 && __popc(equal & ((1u << lane) - 1)) < ties);
        const unsigned pick = __ballot_sync(0xffffffffu, mine && take > 0);
        if (pick >> lane & 1) dst[written + __popc(pick & ((1u << lane) - 1))] = i * 32 + lane;
        written += __popc(pick);
        ties -= min(ties, __popc(equal));
    }
    for (int i = written + lane; i < topk; i += 32) dst[i] = -1;
    if (lane == 0) counts[row] = take;
}

// The same for longer rows: one CTA per row, the keys in shared memory.
__global__ void __launch_bounds__(256) block_topk_cta_kernel(const unsigned long long* __restrict__ keys, int nk, int topk,
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

constexpr int SCORE_SMEM = (128 * SCORE_Q + SCORE_K * K_PITCH) * 8;
constexpr int TOPK_SMEM = 225 * 1024;

}  // namespace

int block_select_max_blocks() { return TOPK_SMEM / 8; }

long long block_select_workspace(int B, int heads, const BlockGrid& g) {
    const long long nq = g.q_blocks(), nk = g.k_blocks();
    return (long long)B * heads * ((nq + nk) * 128 + nq * nk) * 8;
}

cudaError_t init_block_select_attributes() {
    cudaError_t e = cudaFuncSetAttribute(block_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SCORE_SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(block_topk_cta_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TOPK_SMEM);
    return e;
}

cudaError_t launch_block_select(const void* q, long long ldq, const void* k, long long ldk, int B, int heads,
                                const BlockGrid& g, const uint8_t* mask, int topk, int* blocks, int* counts, void* ws,
                                const LaunchCtx& ctx) {
    const int nq = g.q_blocks(), nk = g.k_blocks();
    double* qm = reinterpret_cast<double*>(ws);
    double* km = qm + (long long)B * heads * nq * 128;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(km + (long long)B * heads * nk * 128);
    const int vecs = heads * 16;
    const int threads = vecs < 256 ? (vecs + 31) / 32 * 32 : 256;
    const int slices = (vecs + threads - 1) / threads;
    auto mean = [&](const void* x, long long ld, int n, const int (&d)[3], const int (&b)[3], double* out) {
        block_mean_kernel<<<dim3(n, slices, B), threads, 0, ctx.stream>>>(reinterpret_cast<const __nv_bfloat16*>(x), ld, heads,
                                                                         d[0], d[1], d[2], b[0], b[1], b[2], out);
    };
    mean(q, ldq, nq, g.q, g.qb, qm);
    mean(k, ldk, nk, g.k, g.kb, km);
    block_score_kernel<<<dim3((nk + SCORE_K - 1) / SCORE_K, (nq + SCORE_Q - 1) / SCORE_Q, B * heads), 128, SCORE_SMEM,
                         ctx.stream>>>(qm, km, mask, nq, nk, keys);
    const long long rows = (long long)B * heads * nq;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (nk <= 128)
        block_topk_warp_kernel<4><<<grid, 128, 0, ctx.stream>>>(keys, nk, topk, rows, blocks, counts);
    else if (nk <= 512)
        block_topk_warp_kernel<16><<<grid, 128, 0, ctx.stream>>>(keys, nk, topk, rows, blocks, counts);
    else if (nk <= 1024)
        block_topk_warp_kernel<32><<<grid, 128, 0, ctx.stream>>>(keys, nk, topk, rows, blocks, counts);
    else
        block_topk_cta_kernel<<<(unsigned)rows, 256, nk * 8, ctx.stream>>>(keys, nk, topk, blocks, counts);
    if (ctx.launches) *ctx.launches += 4;
    return cudaGetLastError();
}

}  // namespace wan
