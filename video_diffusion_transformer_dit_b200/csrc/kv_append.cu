// New tokens' keys and values into a paged cache: per token the RMSNorm across
// heads of the key row (optional), its gain, the three-axis rotation at the
// token's place in the sequence, one rounding to bf16, and the store into the
// page that holds the place; the value row is copied; query rows get the same
// norm and rotation into a buffer of their own.
//
// Memory bound: each row is read once and written once, through registers, by 1, 2,
// 4 or 8 warps (up to 6 vectors of 16 bytes per lane).  One row per warp (or warps)
// and then the CTA ends: many short warps hide the chain from the sequence's first
// place over its page to the store better than groups that took several rows each
// with the next row's loads in flight (1.3 times the time).  The k, v and q rows of
// the same tokens follow each other in the grid, so the plain copies of v run beside
// the arithmetic of the other two (k first, then v, then q: 17.7 against 15.6 us), and the
// rows, which nothing reads again, are loaded evict-first so that the gains stay in
// the L1 (without: 18.3).
//   4680 tokens, 12 heads, k, v and q with norm: 15.6 us, 5.5 TB/s; a device copy of
//   the same bytes takes 15.2.  4 x 1560 tokens, 40 heads, two thirds of them there:
//   43.2 us; the copy 37.4.
// Half the vectors per lane and twice the warps (more of them fit in an SM): 16.2
// and 52 us.
//
// A lane's vectors lie 32 apart and a head is 16 vectors, so all of them sit at the
// same place of their head: a lane needs four (cos, sin) pairs.  Where a row has
// several warps its 64 pairs are computed once, through shared memory; a single
// warp computes two per lane and gets the others from the lane 16 further.  The angle
// is taken in turns in fp64, its whole turns dropped, and only the remainder goes to
// fp32 (a position of 1e5 leaves no fraction bits of the angle there).
#include "common.cuh"
#include "kernels.h"

namespace wan {

namespace {

struct AppendParams {
    const __nv_bfloat16 *k, *v, *q;
    long long ldk, ldv, ldq, ldqo;
    __nv_bfloat16* q_out;
    int B, T, heads;
    const int *start, *count;
    const float *k_gain, *q_gain;
    float eps;
    int rope, H, W, zero_rest;
    int nt, nh;             // pairs of the frame and row axes
    KvPages c;
    int log_page;
    uint32_t kinds, rows;   // 2 or 3 (with q); B T
    FastDiv by_T, by_hw, by_W;
    double turns[64];       // theta^(-2 p / width) / (2 pi) of pair p in its axis
};

template <int WPR>
constexpr int WARPS = WPR < 4 ? 4 : WPR;  // per CTA (8 for all: 5 % slower, an SM's room comes free in larger pieces)

// Barrier of a row's warps.  The numbers are immediates: with one from a register a
// CTA is given all 16 barriers, which holds an SM to four CTAs.
template <int WPR, int GROUP = 0>
__device__ __forceinline__ void row_bar(int group) {
    if constexpr (GROUP + 1 < WARPS<WPR> / WPR)
        if (group != GROUP) return row_bar<WPR, GROUP + 1>(group);
    asm volatile("bar.sync %0, %1;" ::"n"(1 + GROUP), "n"(WPR * 32) : "memory");
}

// (cos, sin) of pair `pair` at place (f, ih, iw): the angle in turns
__device__ __forceinline__ float2 rotation(const AppendParams& p, int pair, uint32_t f, uint32_t ih, uint32_t iw) {
    const double turns = (double)(pair < p.nt ? f : pair < p.nt + p.nh ? ih : iw) * p.turns[pair];
    float2 r;
    sincospif(2.0f * (float)(turns - rint(turns)), &r.y, &r.x);
    return r;
}

// grid: {k, v[, q]} fastest, groups of rows; heads * 16 <= 32 NV WPR
template <int NV, int WPR>
__global__ void __launch_bounds__(WARPS<WPR> * 32, 32 / WARPS<WPR>) kv_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ float sums[WARPS<WPR>];
    __shared__ float2 angles[WPR > 1 ? WARPS<WPR> / WPR : 1][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = warp % WPR, group = warp / WPR;
    const int what = blockIdx.x % p.kinds;  // 0 k, 1 v, 2 q
    const int vecs = p.heads * 16;
    const uint32_t row = blockIdx.x / p.kinds * (WARPS<WPR> / WPR) + group;
    if (row >= p.rows) return;
    const int b = p.by_T(row), t = row - b * p.T;
    const int first = __ldg(p.start + b);
    auto vec = [&](int i) { return (i * WPR + sub) * 32 + lane; };
    const uint4* src = reinterpret_cast<const uint4*>(what == 0 ? p.k + row * p.ldk : what == 1 ? p.v + row * p.ldv
                                                                                                : p.q + row * p.ldq);
    uint4 x[NV];
    auto load = [&] {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = vec(i) < vecs ? __ldcs(src + vec(i)) : make_uint4(0, 0, 0, 0);
    };
    if (!p.count) load();  // all rows count: not held up by the sequence's first place
    if (first < 0 || (p.count && t >= __ldg(p.count + b))) {
        if (what == 2 && p.zero_rest) {
            uint4* rest = reinterpret_cast<uint4*>(p.q_out + row * p.ldqo);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (vec(i) < vecs) rest[vec(i)] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    if (p.count) load();
    const uint32_t slot = (uint32_t)first + (uint32_t)t;
    uint4* dst;
    if (what == 2) {
        dst = reinterpret_cast<uint4*>(p.q_out + row * p.ldqo);
    } else {
        const uint32_t at = slot >> p.log_page;
        if (at >= (uint32_t)p.c.max_pages) return;
        const int page = __ldg(p.c.table + (long long)b * p.c.table_ld + at);
        if (page < 0 || page >= p.c.num_pages) return;
        dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(what == 0 ? p.c.k : p.c.v) + page * p.c.page_stride +
                                       (long long)(slot & ((1u << p.log_page) - 1)) * p.c.token_stride);
    }
    if (what == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (vec(i) < vecs) dst[vec(i)] = x[i];
        return;
    }
    // the lane's four rotations: cos and sin of two pairs each
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.rope) {
        const uint32_t hw = (uint32_t)p.H * (uint32_t)p.W;
        const uint32_t f = slot >> 31 ? slot / hw : p.by_hw(slot), in = slot - f * hw;
        const uint32_t ih = p.by_W(in), iw = in - ih * (uint32_t)p.W;
        if (WPR > 1) {
            const int pair = sub * 32 + lane;
            if (pair < 64) angles[group][pair] = rotation(p, pair, f, ih, iw);
        } else {
            const bool upper = lane >= 16;  // this half's two pairs: 0, 1 or 2, 3
            float2 mine[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) mine[i] = rotation(p, (lane & 15) * 4 + (upper ? 2 : 0) + i, f, ih, iw);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float oc = __shfl_xor_sync(0xffffffffu, mine[i].x, 16), os = __shfl_xor_sync(0xffffffffu, mine[i].y, 16);
                cs[i] = upper ? oc : mine[i].x;
                sn[i] = upper ? os : mine[i].y;
                cs[i + 2] = upper ? mine[i].x : oc;
                sn[i + 2] = upper ? mine[i].y : os;
            }
        }
    }
    const float* gain = what == 0 ? p.k_gain : p.q_gain;
    float ss = 0.f;
    if (gain) {
        uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 y = unpack_bf16(w[c]);
                const uint64_t y2 = f2pack(y.x, y.y);
                s2[c & 1] = fma2(y2, y2, s2[c & 1]);
            }
        }
        float a, d;
        f2unpack(add2(s2[0], s2[1]), a, d);
        ss = a + d;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (WPR > 1 && (gain || p.rope)) {  // the row's other warps (the same row, so the same path)
        if (lane == 0) sums[warp] = ss;
        row_bar<WPR>(group);
        ss = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) ss += sums[group * WPR + w];
        if (p.rope) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 r = reinterpret_cast<const float4*>(angles[group])[(lane & 15) * 2 + i];
                cs[2 * i] = r.x;
                sn[2 * i] = r.y;
                cs[2 * i + 1] = r.z;
                sn[2 * i + 1] = r.w;
            }
        }
    }
    if (gain) {  // the norm's factor goes into the rotation
        const float scale = rsqrtf(ss / (float)(p.heads * 128) + p.eps);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            cs[c] *= scale;
            sn[c] *= scale;
        }
    }
    // two pairs at a time: first elements times cos - second ones times sin, and so on
    const uint64_t c2[2] = {f2pack(cs[0], cs[1]), f2pack(cs[2], cs[3])};
    const uint64_t s2[2] = {f2pack(sn[0], sn[1]), f2pack(sn[2], sn[3])};
    const uint64_t m2[2] = {f2pack(-sn[0], -sn[1]), f2pack(-sn[2], -sn[3])};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (vec(i) >= vecs) continue;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float2 y0 = unpack_bf16(w[2 * c]), y1 = unpack_bf16(w[2 * c + 1]);
            if (gain) {
                const float4 g = __ldg(reinterpret_cast<const float4*>(gain) + 2 * vec(i) + c);
                y0.x *= g.x;
                y0.y *= g.y;
                y1.x *= g.z;
                y1.y *= g.w;
            }
            const uint64_t a = f2pack(y0.x, y1.x), d = f2pack(y0.y, y1.y);
            float u0, u1, v0, v1;
            f2unpack(fma2(a, c2[c], mul2(d, m2[c])), u0, u1);
            f2unpack(fma2(a, s2[c], mul2(d, c2[c])), v0, v1);
            o[2 * c] = pack_bf16(u0, v0);  // the one rounding to bf16
            o[2 * c + 1] = pack_bf16(u1, v1);
        }
        dst[vec(i)] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <int NV, int WPR>
void append(const AppendParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.B * p.T, per = WARPS<WPR> / WPR;
    kv_append_kernel<NV, WPR><<<(unsigned)((rows + per - 1) / per) * p.kinds, WARPS<WPR> * 32, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_kv_append(const void* k, long long ldk, const void* v, long long ldv, int B, int T, int heads,
                             const int* start, const int* count, const float* k_gain, float eps, int rope, int H, int W,
                             int rope_t, int rope_h, int rope_w, double theta, const void* q, long long ldq,
                             const float* q_gain, void* q_out, long long ldqo, int zero_rest, const KvPages& c,
                             const LaunchCtx& ctx) {
    AppendParams p{};
    p.k = reinterpret_cast<const __nv_bfloat16*>(k);
    p.v = reinterpret_cast<const __nv_bfloat16*>(v);
    p.q = reinterpret_cast<const __nv_bfloat16*>(q);
    p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
    p.ldk = ldk;
    p.ldv = ldv;
    p.ldq = ldq;
    p.ldqo = ldqo;
    p.B = B;
    p.T = T;
    p.heads = heads;
    p.start = start;
    p.count = count;
    p.k_gain = k_gain;
    p.q_gain = q_gain;
    p.eps = eps;
    p.rope = rope;
    p.zero_rest = zero_rest;
    p.H = H;
    p.W = W;
    p.nt = rope_t / 2;
    p.nh = rope_h / 2;
    p.c = c;
    p.kinds = q ? 3 : 2;
    p.rows = (uint32_t)((long long)B * T);
    p.by_T = fast_div(T);
    p.by_hw = fast_div(rope ? H * W : 1);
    p.by_W = fast_div(rope ? W : 1);
    while ((1 << p.log_page) < c.page_size) ++p.log_page;
    if (rope) {
        const int width[3] = {rope_t, rope_h, rope_w};
        for (int a = 0, n = 0; a < 3; ++a)
            for (int i = 0; i < width[a] / 2; ++i) p.turns[n++] = pow(theta, -2.0 * i / width[a]) * 0.15915494309189533577;
    }
    const int nv = (heads * 16 + 31) / 32;  // vectors per lane of one warp
    if (nv <= 1) append<1, 1>(p, ctx.stream);
    else if (nv <= 3) append<3, 1>(p, ctx.stream);
    else if (nv <= 6) append<6, 1>(p, ctx.stream);
    else if (nv <= 12) append<6, 2>(p, ctx.stream);
    else if (nv <= 20) append<5, 4>(p, ctx.stream);
    else if (nv <= 48) append<6, 8>(p, ctx.stream);
    else return cudaErrorInvalidValue;
    if (ctx.launches) ++*ctx.launches;
    return cudaGetLastError();
}

}  // namespace wan
