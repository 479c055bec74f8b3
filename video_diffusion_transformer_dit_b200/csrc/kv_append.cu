// New tokens' keys and values into a paged cache: per token the RMSNorm across
// heads of the key row (optional), its gain, the three-axis rotation at the
// token's place in the sequence, one rounding to bf16, and the store into the
// page that holds the place; the value row is copied; query rows get the same
// norm and rotation into a buffer of their own.
//
// Memory bound: each row is read once and written once, through registers, by 1, 2,
// 4 or 8 warps (up to 6 vectors of 16 bytes per lane, loaded before anything is
// looked up).  Many short warps hide the chain from the sequence's first place over
// its page to the store; groups that took several rows each, the next row's loads in
// flight and the gains in registers, had a third of the warps and took 1.3 times
// the time.  A lane's vectors lie 32 apart and a head is 16 vectors, so all of them sit at the
// same place of their head: a lane needs four (cos, sin) pairs, computes two and
// gets the others from the lane 16 further.  The angle is taken in turns in fp64,
// its whole turns dropped, and only the remainder goes to fp32 (a position of 1e5
// leaves no fraction bits of the angle there).
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
    double turns[64];       // theta^(-2 p / width) / (2 pi) of pair p in its axis
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = unpack_bf16(w[i]);
        x[2 * i] = p.x;
        x[2 * i + 1] = p.y;
    }
}

// grid: groups of rows x {k, v[, q]}; heads * 16 <= 32 NV WPR
template <int NV, int WPR>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ float sums[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = warp % WPR, group = warp / WPR;
    const int what = blockIdx.y;  // 0 k, 1 v, 2 q
    const int vecs = p.heads * 16;
    const long long row = (long long)blockIdx.x * (8 / WPR) + group;
    if (row >= (long long)p.B * p.T) return;
    const int b = (int)(row / p.T), t = (int)(row - (long long)b * p.T);
    const int first = __ldg(p.start + b);
    auto vec = [&](int i) { return (i * WPR + sub) * 32 + lane; };
    if (first < 0 || (p.count && t >= __ldg(p.count + b))) {
        if (what == 2 && p.zero_rest) {
            uint4* rest = reinterpret_cast<uint4*>(p.q_out + row * p.ldqo);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (vec(i) < vecs) rest[vec(i)] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const uint4* src = reinterpret_cast<const uint4*>(what == 0 ? p.k + row * p.ldk : what == 1 ? p.v + row * p.ldv
                                                                                                : p.q + row * p.ldq);
    uint4 x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = vec(i) < vecs ? src[vec(i)] : make_uint4(0, 0, 0, 0);
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
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    if (p.rope) {
        const uint32_t hw = (uint32_t)p.H * (uint32_t)p.W;
        const uint32_t f = slot / hw, in = slot - f * hw, ih = in / (uint32_t)p.W, iw = in - ih * (uint32_t)p.W;
        const bool upper = lane >= 16;  // this half's two pairs: 0, 1 or 2, 3
        float c2[2], s2[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pair = (lane & 15) * 4 + (upper ? 2 : 0) + i;
            const uint32_t pos = pair < p.nt ? f : pair < p.nt + p.nh ? ih : iw;
            const double turns = (double)pos * p.turns[pair];
            sincospif(2.0f * (float)(turns - rint(turns)), &s2[i], &c2[i]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float oc = __shfl_xor_sync(0xffffffffu, c2[i], 16), os = __shfl_xor_sync(0xffffffffu, s2[i], 16);
            cs[i] = upper ? oc : c2[i];
            sn[i] = upper ? os : s2[i];
            cs[i + 2] = upper ? c2[i] : oc;
            sn[i + 2] = upper ? s2[i] : os;
        }
    }
    const float* gain = what == 0 ? p.k_gain : p.q_gain;
    float scale = 1.0f;
    if (gain) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float y[8];
            unpack8(x[i], y);
#pragma unroll
            for (int c = 0; c < 8; ++c) ss += y[c] * y[c];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (WPR > 1) {  // the row's other warps (the same row, so the same path)
            if (lane == 0) sums[warp] = ss;
            named_bar(1 + group, WPR * 32);
            ss = 0.f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) ss += sums[group * WPR + w];
        }
        scale = rsqrtf(ss / (float)(p.heads * 128) + p.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (vec(i) >= vecs) continue;
        float y[8];
        unpack8(x[i], y);
        if (gain) {
            const float4 g0 = __ldg(reinterpret_cast<const float4*>(gain) + 2 * vec(i));
            const float4 g1 = __ldg(reinterpret_cast<const float4*>(gain) + 2 * vec(i) + 1);
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
            for (int c = 0; c < 8; ++c) y[c] = y[c] * scale * g[c];
        }
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)  // the one rounding to bf16
            o[c] = pack_bf16(y[2 * c] * cs[c] - y[2 * c + 1] * sn[c], y[2 * c] * sn[c] + y[2 * c + 1] * cs[c]);
        dst[vec(i)] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <int NV, int WPR>
void append(const AppendParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.B * p.T, per = 8 / WPR;
    kv_append_kernel<NV, WPR><<<dim3((unsigned)((rows + per - 1) / per), p.q ? 3 : 2), 256, 0, stream>>>(p);
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
