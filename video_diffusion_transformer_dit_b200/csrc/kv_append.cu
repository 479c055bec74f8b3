// New tokens' keys and values into a paged cache: per token the RMSNorm across
// heads of the key row (optional), its gain, the three-axis rotation at the
// token's place in the sequence, one rounding to bf16, and the store into the
// page that holds the place; the value row is copied; query rows get the same
// norm and rotation into a buffer of their own.
//
// Memory bound: each row is read once and written once.  One warp per row; a
// lane's 16-byte vectors are lane, lane + 32, ..., and since a head is 16
// vectors all of them sit at the same place of their head, so a lane needs four
// (cos, sin) pairs in all and computes them itself: the angle and its remainder
// by 2 pi in fp64 (a position of 1e5 leaves no fraction bits of the angle in
// fp32), cos and sin of the remainder in fp32.
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
    int rope, H, W;
    int nt, nh;             // pairs of the frame and row axes
    KvPages c;
    double freq[64];        // theta^(-2 p / width) of pair p in its axis
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

// grid: rows / 8 x {k, v[, q]}
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendParams p) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.B * p.T) return;
    const int b = (int)(row / p.T), t = (int)(row % p.T);
    if (p.count && t >= __ldg(p.count + b)) return;
    const int first = __ldg(p.start + b);
    const long long slot = (long long)first + t;
    const int what = blockIdx.y;  // 0 k, 1 v, 2 q
    const int vecs = p.heads * 16;
    const __nv_bfloat16* src = what == 0 ? p.k + row * p.ldk : what == 1 ? p.v + row * p.ldv : p.q + row * p.ldq;
    __nv_bfloat16* dst;
    if (what == 2) {
        if (first < 0) return;
        dst = p.q_out + row * p.ldqo;
    } else {
        const long long at = slot / p.c.page_size;
        if (first < 0 || at >= p.c.max_pages) return;
        const int page = __ldg(p.c.table + (long long)b * p.c.table_ld + at);
        if (page < 0 || page >= p.c.num_pages) return;
        dst = reinterpret_cast<__nv_bfloat16*>(what == 0 ? p.c.k : p.c.v) + page * p.c.page_stride +
              (slot - at * p.c.page_size) * p.c.token_stride;
    }
    if (what == 1) {
        for (int i = lane; i < vecs; i += 32)
            reinterpret_cast<uint4*>(dst)[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
        return;
    }
    const float* gain = what == 0 ? p.k_gain : p.q_gain;
    float scale = 1.0f;
    if (gain) {
        float ss = 0.f;
        for (int i = lane; i < vecs; i += 32) {
            float x[8];
            unpack8(reinterpret_cast<const uint4*>(src)[i], x);
#pragma unroll
            for (int c = 0; c < 8; ++c) ss += x[c] * x[c];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        scale = rsqrtf(ss / (float)(p.heads * 128) + p.eps);
    }
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    if (p.rope) {
        const long long hw = (long long)p.H * p.W;
        const long long f = slot / hw;
        const int in = (int)(slot - f * hw), ih = in / p.W, iw = in - ih * p.W;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pair = (lane & 15) * 4 + i;
            const double pos = pair < p.nt ? (double)f : pair < p.nt + p.nh ? (double)ih : (double)iw;
            const double angle = pos * p.freq[pair];
            const double turns = rint(angle * 0.15915494309189535);  // 1 / (2 pi)
            sincosf((float)fma(turns, -6.283185307179586, angle), &sn[i], &cs[i]);
        }
    }
    for (int i = lane; i < vecs; i += 32) {
        float x[8];
        unpack8(reinterpret_cast<const uint4*>(src)[i], x);
        if (gain) {
            const float4 g0 = __ldg(reinterpret_cast<const float4*>(gain) + 2 * i);
            const float4 g1 = __ldg(reinterpret_cast<const float4*>(gain) + 2 * i + 1);
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] = x[c] * scale * g[c];
        }
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            o[c] = pack_bf16(x[2 * c] * cs[c] - x[2 * c + 1] * sn[c], x[2 * c] * sn[c] + x[2 * c + 1] * cs[c]);
        reinterpret_cast<uint4*>(dst)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

cudaError_t launch_kv_append(const void* k, long long ldk, const void* v, long long ldv, int B, int T, int heads,
                             const int* start, const int* count, const float* k_gain, float eps, int rope, int H, int W,
                             int rope_t, int rope_h, int rope_w, double theta, const void* q, long long ldq,
                             const float* q_gain, void* q_out, long long ldqo, const KvPages& c, const LaunchCtx& ctx) {
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
    p.H = H;
    p.W = W;
    p.nt = rope_t / 2;
    p.nh = rope_h / 2;
    p.c = c;
    if (rope) {
        const int width[3] = {rope_t, rope_h, rope_w};
        for (int a = 0, n = 0; a < 3; ++a)
            for (int i = 0; i < width[a] / 2; ++i) p.freq[n++] = pow(theta, -2.0 * i / width[a]);
    }
    const dim3 grid((unsigned)(((long long)B * T + 7) / 8), q ? 3 : 2);
    kv_append_kernel<<<grid, 256, 0, ctx.stream>>>(p);
    if (ctx.launches) ++*ctx.launches;
    return cudaGetLastError();
}

}  // namespace wan
