// Attention over listed parts of the sequence, head_dim 128, bf16 operands,
// fp32 softmax:
//   blocks  each query block (a box of up to 128 tokens of the query grid)
//           attends to the key blocks listed for it (boxes of 16..128 tokens);
//   pages   the T new tokens of each sequence attend to the sequence's cached
//           keys and values, which lie in pages of 16..128 tokens.
// Both are the same loop: a list of token groups, gathered by TMA into tiles of
// 128 keys, softmax with a running maximum and sum, O += P V per tile.
//
// A work unit is one query tile (up to 128 rows of one head and sample) and one
// split of its list.  A CTA (one per SM) carries two units side by side
// (streams t = 0, 1), each with its own Q tile, S_t, P_t (over S_t) and O_t in
// tensor memory, so one stream's exponentials overlap the other's MMAs although
// the two read different keys.  In step k of its unit a stream issues
// S(k) = Q K_k^T and then O += P(k-1) V_(k-1); the streams alternate step by
// step, and their K and V tiles pass through one ring of five 32 KB slots in
// that order.  Streams walk units blockIdx.x * 2 + t, + 2 * gridDim.x, ...
//
// Warps (registers per thread as in the dense kernel):
//   0      TMA producer (whole warp: each lane gathers one token group of the
//          tile) and the 128-bit mask of the tile's keys;
//   1      tensor-memory owner and MMA issuer; it also zeroes the V rows of a tile
//          past the sequence's end inside a page before the tile's P.V;
//   2..3   idle;
//   4..11  softmax of stream 0 / 1, one query row per thread; warps without a
//          row only keep the barriers' counts.
// Where there are too few query tiles to fill the GPU, lists are split: each
// split writes its normalised fp32 rows and their log-sum-exp, and
// list_join_kernel joins them.
#include "common.cuh"
#include "kernels.h"

namespace wan {

namespace alist {
constexpr int TILE_BYTES = 128 * 128 * 2;  // 128 rows x 128 columns: two 64-column swizzled halves
constexpr int HALF_BYTES = 128 * 128;
constexpr int SLOTS = 5;
constexpr int MASKS = 8;                   // key masks per stream (tiles in flight: at most 4)
constexpr int SQ = 0;
constexpr int SKV = SQ + 2 * TILE_BYTES;
constexpr int SMASK = SKV + SLOTS * TILE_BYTES;
constexpr int SBAR = SMASK + 2 * MASKS * 16;
constexpr int SMEM_BYTES = SBAR + 256 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
constexpr int THREADS = 384;
constexpr int REGS_LAUNCH = 168;
constexpr int REGS_CONTROL = 104;
constexpr int REGS_SOFTMAX = 192;
static_assert(128 * REGS_CONTROL + 256 * REGS_SOFTMAX <= THREADS * REGS_LAUNCH, "register split");
constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units
constexpr int PLAN_SMS = 148;              // SMs the split plan assumes
enum Mode { BLOCKS, PAGES };
}  // namespace alist

struct ListParams {
    int units, splits, nqb, heads, B;
    int rows;               // rows of a full query tile
    int E, log_group;       // token groups per tile, log2 of tokens per group
    // blocks
    BlockGrid g;
    const int* blocks;
    const int* counts;
    int topk, nkb;
    // pages
    const int* table;
    long long table_ld;
    const int* lens;
    int max_pages, num_pages, T;
    __nv_bfloat16* o;
    long long ldo;
    float* lse;             // [B, heads, query tokens] or null
    float* part_o;          // [unit][rows][128] fp32 (splits > 1)
    float* part_lse;        // [unit][rows], log2 units
    float scale_log2;
    WaitCtl wc;
};

// One unit: its head, sample, query tile and the tiles [j0, j0 + n) of its list.
struct ListUnit {
    int b, h, qt, j0, n;
    int length;             // groups in the list (blocks) or tokens in the cache (pages)
    bool dirty;             // pages: the last tile ends inside a page
};

template <alist::Mode MODE>
__device__ __forceinline__ ListUnit list_unit(const ListParams& p, int u) {
    ListUnit x;
    // splits slowest: CTAs that run together read the same tokens of several heads
    const int per = p.nqb * p.heads * p.B;
    const int s = u / per;
    int r = u - s * per;
    x.qt = r % p.nqb;
    r /= p.nqb;
    x.h = r % p.heads;
    x.b = r / p.heads;
    int tiles;
    if (MODE == alist::BLOCKS) {
        const int c = __ldg(p.counts + ((long long)x.b * p.heads + x.h) * p.nqb + x.qt);
        x.length = min(max(c, 0), p.topk);
        tiles = (x.length + p.E - 1) / p.E;
    } else {
        const int cap = p.max_pages << p.log_group;
        x.length = min(max(__ldg(p.lens + x.b), 0), cap);
        tiles = (x.length + 127) >> 7;
    }
    x.j0 = (int)((long long)tiles * s / p.splits);
    const int j1 = (int)((long long)tiles * (s + 1) / p.splits);
    x.n = j1 - x.j0;
    x.dirty = MODE == alist::PAGES && j1 == tiles && (x.length & ((1 << p.log_group) - 1)) != 0;
    return x;
}

// The interleaved walk that producer and issuer share: step k
// of a unit loads K(k) (k < n) and V(k - 1) (k > 0); empty units have no step.
template <alist::Mode MODE>
struct ListWalk {
    ListUnit x;
    int u, k;
    __device__ __forceinline__ void start(const ListParams& p, int t) {
        u = blockIdx.x * 2 + t - 2 * gridDim.x;
        next(p);
    }
    __device__ __forceinline__ void next(const ListParams& p) {
        k = 0;
        do {
            u += 2 * gridDim.x;
            if (u >= p.units) return;
            x = list_unit<MODE>(p, u);
        } while (x.n == 0);
    }
    __device__ __forceinline__ bool live(const ListParams& p) const { return u < p.units; }
};

// Origin of a token group: block (f, i, j) or page number (in f); out-of-range
// batch / page coordinates where there is none (TMA fills zeros).
struct ListGroup {
    int f, i, j, b;
    bool ok;
};

template <alist::Mode MODE>
__global__ void __launch_bounds__(alist::THREADS, 1)
    attn_list_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ListParams p) {
    using namespace alist;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint4* masks = reinterpret_cast<uint4*>(smem + SMASK);  // [2][MASKS]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SBAR);
    uint64_t* q_full = bars;                 // [2]
    uint64_t* q_empty = q_full + 2;          // [2] the unit's last S has read Q
    uint64_t* kv_full = q_empty + 2;         // [SLOTS]
    uint64_t* kv_empty = kv_full + SLOTS;    // [SLOTS]
    uint64_t* s_full = kv_empty + SLOTS;     // [2]
    uint64_t* s_read = s_full + 2;           // [2] the softmax has read S_t
    uint64_t* p_part = s_read + 2;           // [2] P of keys 0..63 stored
    uint64_t* p_full = p_part + 2;           // [2]
    uint64_t* o_final = p_full + 2;          // [2]
    uint64_t* drain = o_final + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full + t, 1);
            mbar_init(q_empty + t, 1);
            mbar_init(s_full + t, 1);
            mbar_init(s_read + t, 4);
            mbar_init(p_part + t, 4);
            mbar_init(p_full + t, 4);
            mbar_init(o_final + t, 1);
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(kv_full + s, 1);
            mbar_init(kv_empty + s, 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // producer: slots with a load issued and the phase it completes; Q phases;
    // issuer: whether any MMA went out (both drained after an abort, before exit)
    uint32_t armed = 0, par = 0;
    int qpar[2] = {-1, -1};
    bool issued = false;

    if (warp < 4) {
        regs_dealloc<REGS_CONTROL>();
        if (warp == 0) {
            // ---------------- producer ----------------
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                int r = 1;
                if (lane == 0) r = mbar_wait(bar, parity, abort_flag, p.wc) ? 1 : 0;
                return __shfl_sync(0xffffffffu, r, 0) != 0;
            };
            const int group = 1 << p.log_group;
            // place of the lane's four key columns inside their group
            int off[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int r = (c * 32 + lane) & (group - 1);
                off[c] = r;
                if (MODE == BLOCKS) {
                    const int dj = r % p.g.kb[2], di = (r / p.g.kb[2]) % p.g.kb[1], df = r / (p.g.kb[2] * p.g.kb[1]);
                    off[c] = df | di << 8 | dj << 16;
                }
            }
            auto group_at = [&](const ListUnit& x, int j) -> ListGroup {  // lane e: group e of tile j
                ListGroup o{0, 0, 0, MODE == BLOCKS ? p.B : p.num_pages, false};
                const int idx = j * p.E + lane;
                if (lane >= p.E) return o;
                if (MODE == BLOCKS) {
                    if (idx >= x.length) return o;
                    const int id = __ldg(p.blocks + (((long long)x.b * p.heads + x.h) * p.nqb + x.qt) * p.topk + idx);
                    if (id < 0 || id >= p.nkb) return o;
                    const int nj = p.g.nk(2), ni = p.g.nk(1);
                    const int r = id / nj;
                    o.j = (id - r * nj) * p.g.kb[2];
                    o.i = (r % ni) * p.g.kb[1];
                    o.f = (r / ni) * p.g.kb[0];
                    o.b = x.b;
                    o.ok = true;
                } else {
                    if ((idx << p.log_group) >= x.length) return o;
                    const int page = __ldg(p.table + (long long)x.b * p.table_ld + idx);
                    if (page < 0 || page >= p.num_pages) return o;
                    o.b = page;
                    o.f = idx << p.log_group;  // first token
                    o.ok = true;
                }
                return o;
            };
            auto write_mask = [&](const ListUnit& x, const ListGroup& o, uint4* dst) {
                uint32_t w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int e = (c * 32 + lane) >> p.log_group;
                    const bool ok = __shfl_sync(0xffffffffu, (int)o.ok, e) != 0;
                    const int f = __shfl_sync(0xffffffffu, o.f, e);
                    bool in;
                    if (MODE == BLOCKS) {
                        const int i = __shfl_sync(0xffffffffu, o.i, e), j = __shfl_sync(0xffffffffu, o.j, e);
                        in = ok && f + (off[c] & 255) < p.g.k[0] && i + (off[c] >> 8 & 255) < p.g.k[1] &&
                             j + (off[c] >> 16) < p.g.k[2];
                    } else {
                        in = ok && f + off[c] < x.length;
                    }
                    w[c] = __ballot_sync(0xffffffffu, in);
                }
                if (lane == 0) *dst = make_uint4(w[0], w[1], w[2], w[3]);
            };
            int c = 0;  // loads so far
            auto load = [&](const CUtensorMap* tm, const ListUnit& x, const ListGroup& o) -> bool {
                const int slot = c % SLOTS;
                const uint32_t phase = (c / SLOTS) & 1;
                ++c;
                if (!wait(kv_empty + slot, phase ^ 1)) return false;
                if (lane == 0) mbar_expect_tx(kv_full + slot, TILE_BYTES);
                __syncwarp();
                if (lane < p.E) {
                    uint8_t* dst = smem + SKV + slot * TILE_BYTES + (lane << p.log_group) * 128;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (MODE == BLOCKS)
                            tma_load_5d(dst + half * HALF_BYTES, tm, kv_full + slot, x.h * 128 + half * 64, o.j, o.i, o.f, o.b);
                        else
                            tma_load_3d(dst + half * HALF_BYTES, tm, kv_full + slot, x.h * 128 + half * 64, 0, o.b);
                    }
                }
                armed |= 1u << slot;
                par = (par & ~(1u << slot)) | phase << slot;
                return true;
            };
            ListWalk<MODE> w[2];
            ListGroup last[2];   // the previous tile's groups: its V goes one step after its K
            int tiles[2] = {0, 0}, unit[2] = {0, 0};
            bool ok = true;
            for (int t = 0; t < 2; ++t) w[t].start(p, t);
            while (ok && (w[0].live(p) || w[1].live(p))) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || !w[t].live(p)) continue;
                    const int k = w[t].k;
                    if (k == 0) {
                        if (!wait(q_empty + t, (unit[t] & 1) ^ 1)) { ok = false; continue; }
                        if (lane == 0) {
                            uint8_t* dst = smem + SQ + t * TILE_BYTES;
                            const int h0 = w[t].x.h * 128;
                            if (MODE == BLOCKS) {
                                const int nj = p.g.nq(2), ni = p.g.nq(1), qt = w[t].x.qt;
                                const int j = (qt % nj) * p.g.qb[2], i = (qt / nj % ni) * p.g.qb[1], f = (qt / nj / ni) * p.g.qb[0];
                                mbar_expect_tx(q_full + t, p.rows * 256);
                                tma_load_5d(dst, &tmQ, q_full + t, h0, j, i, f, w[t].x.b);
                                tma_load_5d(dst + HALF_BYTES, &tmQ, q_full + t, h0 + 64, j, i, f, w[t].x.b);
                            } else {
                                mbar_expect_tx(q_full + t, TILE_BYTES);
                                tma_load_3d(dst, &tmQ, q_full + t, h0, w[t].x.qt * 128, w[t].x.b);
                                tma_load_3d(dst + HALF_BYTES, &tmQ, q_full + t, h0 + 64, w[t].x.qt * 128, w[t].x.b);
                            }
                        }
                        qpar[t] = unit[t] & 1;
                        ++unit[t];
                    }
                    const ListGroup prev = last[t];
                    if (k < w[t].x.n) {
                        last[t] = group_at(w[t].x, w[t].x.j0 + k);
                        write_mask(w[t].x, last[t], masks + t * MASKS + (tiles[t] & (MASKS - 1)));
                        ++tiles[t];
                        ok = load(&tmK, w[t].x, last[t]);
                    }
                    if (ok && k > 0) ok = load(&tmV, w[t].x, prev);
                    if (++w[t].k > w[t].x.n) w[t].next(p);
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer ----------------
            // the whole warp runs the loop; lane 0 waits, one elected lane issues
            constexpr uint32_t ID_QK = idesc_bf16(128, 128, false);
            constexpr uint32_t ID_QK64 = idesc_bf16(128, 64, false);
            constexpr uint32_t ID_PV = idesc_bf16(128, 128, true);
            const uint64_t dq = sdesc_kmajor_sw128(smem_u32(smem + SQ));
            const uint64_t dk = sdesc_kmajor_sw128(smem_u32(smem + SKV));
            const uint64_t dv = sdesc_mnmajor_sw128(smem_u32(smem + SKV), HALF_BYTES);
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                int r = 1;
                if (lane == 0) r = mbar_spin(bar, parity, abort_flag, p.wc) ? 1 : 0;
                return __shfl_sync(0xffffffffu, r, 0) != 0;
            };
            // S_t = Q_t K^T: all 128 keys, keys 64..127 (columns P does not
            // occupy) or keys 0..63 (after the P.V that reads P there)
            enum { S_ALL, S_HI, S_LO };
            auto issue_s = [&](int t, int slot, bool last, int part) {
                tc_fence_after();
                const uint64_t a = dq + (uint64_t)((t * TILE_BYTES) >> 4);
                const uint64_t b = dk + (uint64_t)((slot * TILE_BYTES + (part == S_HI ? 64 * 128 : 0)) >> 4);
                const uint32_t d = tmem + t * 128 + (part == S_HI ? 64 : 0);
                const uint32_t idesc = part == S_ALL ? ID_QK : ID_QK64;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t o = ((kk >> 2) * HALF_BYTES + (kk & 3) * 32) >> 4;
                        umma_bf16_ss(d, a + o, b + o, idesc, kk != 0);
                    }
                    if (part != S_HI) {
                        umma_commit(s_full + t);
                        umma_commit(kv_empty + slot);
                        if (last) umma_commit(q_empty + t);
                    }
                }
                __syncwarp();
                issued = true;
            };
            // one K = 64 half of O_t += P_t V, P_t read from the S_t columns
            auto issue_pv = [&](int t, int slot, bool first, bool last, int half) {
                tc_fence_after();
                const uint64_t b = dv + (uint64_t)((slot * TILE_BYTES) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                        umma_bf16_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, b + ((kk * 2048) >> 4), ID_PV,
                                     !(first && kk == 0));
                    if (half == 1) {
                        umma_commit(kv_empty + slot);
                        if (last) umma_commit(o_final + t);
                    }
                }
                __syncwarp();
            };
            ListWalk<MODE> w[2];
            int c = 0, tiles[2] = {0, 0}, unit[2] = {0, 0};
            bool ok = true;
            for (int t = 0; t < 2; ++t) w[t].start(p, t);
            while (ok && (w[0].live(p) || w[1].live(p))) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || !w[t].live(p)) continue;
                    const int k = w[t].k, n = w[t].x.n;
                    const int sk = c % SLOTS;  // slot of K(k)
                    const bool more = k < n, last_s = k == n - 1;
                    if (more) {
                        const uint32_t phase = (c / SLOTS) & 1;
                        ++c;
                        if (k == 0) {
                            if (!wait(q_full + t, unit[t] & 1) || !wait(kv_full + sk, phase)) { ok = false; continue; }
                            issue_s(t, sk, last_s, S_ALL);
                            ++unit[t];
                        } else {
                            if (!wait(s_read + t, (tiles[t] - 1) & 1) || !wait(kv_full + sk, phase)) { ok = false; continue; }
                            issue_s(t, sk, last_s, S_HI);
                        }
                    }
                    if (k > 0) {
                        const int sv = c % SLOTS;
                        const uint32_t phase = (c / SLOTS) & 1;
                        ++c;
                        const uint32_t tp = (tiles[t] - 1) & 1;  // phase of tile k - 1
                        if (!wait(kv_full + sv, phase)) { ok = false; continue; }
                        if (MODE == PAGES && k == n && w[t].x.dirty) {
                            // rows past the sequence hold foreign memory: 0 * NaN would reach O
                            const int valid = w[t].x.length - (w[t].x.j0 + n - 1) * 128;  // 1..127
                            const uint32_t base = smem_u32(smem + SKV + sv * TILE_BYTES);
                            for (int i = valid * 8 + lane; i < 1024; i += 32) {
                                st_shared_v4(base + i * 16, 0, 0, 0, 0);
                                st_shared_v4(base + HALF_BYTES + i * 16, 0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        if (!wait(p_part + t, tp)) { ok = false; continue; }
                        issue_pv(t, sv, k == 1, false, 0);
                        if (!wait(p_full + t, tp)) { ok = false; continue; }
                        issue_pv(t, sv, false, k == n, 1);
                        if (more) issue_s(t, sk, last_s, S_LO);
                    }
                    if (more) ++tiles[t];
                    if (++w[t].k > n) w[t].next(p);
                }
            }
        }
    } else {
        regs_alloc<REGS_SOFTMAX>();
        // ---------------- softmax / output warps ----------------
        const int t = (warp - 4) >> 2;
        const int qq = warp & 3;                         // TMEM lane quarter
        const int r = qq * 32 + lane;                    // row inside the tile == TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(qq * 32) << 16;
        const uint32_t TS = tmem + t * 128 + lane_off;   // S_t (and P_t)
        const uint32_t TO = tmem + 256 + t * 128 + lane_off;
        const int Lq = MODE == BLOCKS ? p.g.q_tokens() : p.T;
        bool ok = true;
        int g = 0, iu = 0;  // tiles and non-empty units so far
        for (int u = blockIdx.x * 2 + t; ok && u < p.units; u += 2 * gridDim.x) {
            const ListUnit x = list_unit<MODE>(p, u);
            // query token of this thread's row, -1 for none
            int token = -1;
            if (MODE == BLOCKS) {
                const int nj = p.g.nq(2), ni = p.g.nq(1);
                const int f = (x.qt / nj / ni) * p.g.qb[0] + r / (p.g.qb[2] * p.g.qb[1]);
                const int i = (x.qt / nj % ni) * p.g.qb[1] + r / p.g.qb[2] % p.g.qb[1];
                const int j = (x.qt % nj) * p.g.qb[2] + r % p.g.qb[2];
                if (r < p.rows && f < p.g.q[0] && i < p.g.q[1] && j < p.g.q[2]) token = (f * p.g.q[1] + i) * p.g.q[2] + j;
            } else if (x.qt * 128 + r < p.T) {
                token = x.qt * 128 + r;
            }
            const bool active = __any_sync(0xffffffffu, token >= 0);
            float m_run = -INFINITY, l_run = 0.0f;
            for (int j = 0; j < x.n; ++j, ++g) {
                // all tcgen05.ld/st below are warp-collective: the warp's decisions stay uniform
                if (!__all_sync(0xffffffffu, mbar_wait(s_full + t, g & 1, abort_flag, p.wc))) { ok = false; break; }
                tc_fence_after();
                if (!active) {  // no row here: the S columns stay as they are, nothing reads their product
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(s_read + t);
                        mbar_arrive(p_part + t);
                        mbar_arrive(p_full + t);
                    }
                    continue;
                }
                uint32_t sv[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(TS + c * 32, sv[c]);
                const uint4 mk = masks[t * MASKS + (g & (MASKS - 1))];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld_wait(sv[c]);
                {  // S_t is in registers: the MMA may rewrite its upper key half
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_read + t);
                }
                const uint32_t mw[4] = {mk.x, mk.y, mk.z, mk.w};
                if ((mw[0] & mw[1] & mw[2] & mw[3]) != 0xffffffffu) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(mw[c] >> i & 1)) sv[c][i] = __float_as_uint(-INFINITY);
                }
                // row maximum: eight independent 3-input max chains
                float mx[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t* v = &sv[q >> 1][(q & 1) * 16];
                    float a = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
                    for (int i = 2; i < 16; i += 2) a = max3f(a, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                    mx[q] = a;
                }
                const float m_tile =
                    max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * p.scale_log2;
                const float m_new = fmaxf(m_run, m_tile);
                const bool rescale = m_new > m_run + RESCALE_THRESHOLD;
                const float m_use = rescale ? m_new : m_run;
                const float m_sub = m_use == -INFINITY ? 0.0f : m_use;  // every key so far masked: all exponentials are 0
                // O_t is idle here (the commit of S_t also covered the previous P_t V) and
                // must be rescaled before the first half of this tile's P_t V is issued
                const float alpha = rescale ? ex2_approx(m_run - m_use) : 1.0f;  // 0 on the first tile
                if (j > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t ov[32];
                        tmem_ld32(TO + c * 32, ov);
                        tmem_ld_wait(ov);
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tmem_st32(TO + c * 32, ov);
                    }
                }
                // probabilities on packed fp32 pairs, summed in fp32 and rounded to bf16 (the
                // tensor core's operand type: half a step is 2^-9 of each) over their S columns
                uint64_t ps2[2] = {0ull, 0ull};
                const uint64_t scale2 = f2pack(p.scale_log2, p.scale_log2);
                const uint64_t negm2 = f2pack(-m_sub, -m_sub);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pc[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const uint64_t x2 = fma2(f2pack(__uint_as_float(sv[c][i]), __uint_as_float(sv[c][i + 1])), scale2, negm2);
                        float x0, x1;
                        f2unpack(x2, x0, x1);
                        const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
                        ps2[(i >> 1) & 1] = add2(ps2[(i >> 1) & 1], f2pack(e0, e1));
                        pc[i / 2] = pack_bf16(e0, e1);
                    }
                    tmem_st16(TS + c * 16, pc);
                    if (c == 1) {  // keys 0..63 (and any O rescale) stored: their P.V may start
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_part + t);
                    }
                }
                float ps[4];
                f2unpack(ps2[0], ps[0], ps[1]);
                f2unpack(ps2[1], ps[2], ps[3]);
                tmem_st_wait();
                if (rescale) {
                    l_run *= alpha;
                    m_run = m_use;
                }
                l_run += (ps[0] + ps[1]) + (ps[2] + ps[3]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + t);
            }
            if (!ok) break;
            // the unit's output: O_t / l once its last P.V has landed (zero rows where no key was left)
            if (x.n > 0) {
                if (!__all_sync(0xffffffffu, mbar_wait(o_final + t, iu & 1, abort_flag, p.wc))) { ok = false; break; }
                ++iu;
                tc_fence_after();
            }
            if (!active) continue;
            const bool none = l_run == 0.0f;
            const float inv = none ? 0.0f : 1.0f / l_run;
            const float lse2 = none ? -INFINITY : m_run + log2f(l_run);
            const bool direct = p.splits == 1;
            if (token >= 0) {
                if (!direct)
                    p.part_lse[(long long)u * p.rows + r] = lse2;
                else if (p.lse)
                    p.lse[((long long)x.b * p.heads + x.h) * Lq + token] = lse2 * 0.6931471805599453f;
            }
            if (!direct && x.n == 0) continue;  // the join does not read rows whose sum is empty
            __nv_bfloat16* orow = p.o + ((long long)x.b * Lq + token) * p.ldo + x.h * 128;
            float* prow = p.part_o + ((long long)u * p.rows + r) * 128;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t ov[32];
                if (x.n > 0) {
                    tmem_ld32(TO + c * 32, ov);
                    tmem_ld_wait(ov);
                }
                if (none) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) ov[i] = 0;
                }
                if (token >= 0 && direct) {
                    uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        dst[w] = make_uint4(pack_bf16(__uint_as_float(ov[8 * w]) * inv, __uint_as_float(ov[8 * w + 1]) * inv),
                                            pack_bf16(__uint_as_float(ov[8 * w + 2]) * inv, __uint_as_float(ov[8 * w + 3]) * inv),
                                            pack_bf16(__uint_as_float(ov[8 * w + 4]) * inv, __uint_as_float(ov[8 * w + 5]) * inv),
                                            pack_bf16(__uint_as_float(ov[8 * w + 6]) * inv, __uint_as_float(ov[8 * w + 7]) * inv));
                } else if (token >= 0) {
                    float4* dst = reinterpret_cast<float4*>(prow + c * 32);
#pragma unroll
                    for (int w = 0; w < 8; ++w)
                        dst[w] = make_float4(__uint_as_float(ov[4 * w]) * inv, __uint_as_float(ov[4 * w + 1]) * inv,
                                             __uint_as_float(ov[4 * w + 2]) * inv, __uint_as_float(ov[4 * w + 3]) * inv);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a wait gave up somewhere in the CTA: let this CTA's own loads and MMAs
        // land (bounded) before its shared and tensor memory are released
        if (warp == 0 && lane == 0) {
            for (int t = 0; t < 2; ++t)
                if (qpar[t] >= 0) mbar_drain(q_full + t, static_cast<uint32_t>(qpar[t]), 200000000ull);
            for (int s = 0; s < SLOTS; ++s)
                if (armed & (1u << s)) mbar_drain(kv_full + s, (par >> s) & 1, 200000000ull);
        } else if (warp == 1 && issued) {
            if (elect_one()) {  // the lane that issued the MMAs
                umma_commit(drain);
                mbar_drain(drain, 0, 200000000ull);
            }
            __syncwarp();
        }
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the splits of one query row: O = sum_s w_s O_s, w_s = 2^(lse_s - lse).
// One warp per row; a split without keys has lse -inf and is not read.
template <alist::Mode MODE>
__global__ void __launch_bounds__(256) list_join_kernel(const __grid_constant__ ListParams p) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int per = p.nqb * p.heads * p.B;
    if (row >= (long long)per * p.rows) return;
    const int unit = (int)(row / p.rows), r = (int)(row % p.rows);
    const int qt = unit % p.nqb, h = unit / p.nqb % p.heads, b = unit / p.nqb / p.heads;
    int token, Lq;
    if (MODE == alist::BLOCKS) {
        const int nj = p.g.nq(2), ni = p.g.nq(1);
        const int f = (qt / nj / ni) * p.g.qb[0] + r / (p.g.qb[2] * p.g.qb[1]);
        const int i = (qt / nj % ni) * p.g.qb[1] + r / p.g.qb[2] % p.g.qb[1];
        const int j = (qt % nj) * p.g.qb[2] + r % p.g.qb[2];
        if (f >= p.g.q[0] || i >= p.g.q[1] || j >= p.g.q[2]) return;
        token = (f * p.g.q[1] + i) * p.g.q[2] + j;
        Lq = p.g.q_tokens();
    } else {
        token = qt * 128 + r;
        Lq = p.T;
        if (token >= Lq) return;
    }
    auto at = [&](int s) { return ((long long)s * per + unit) * p.rows + r; };
    float m = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) m = fmaxf(m, p.part_lse[at(s)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    for (int s = 0; s < p.splits; ++s) {
        const float l = p.part_lse[at(s)];
        if (l == -INFINITY) continue;
        const float w = exp2f(l - m);
        const float4 x = *reinterpret_cast<const float4*>(p.part_o + at(s) * 128 + lane * 4);
        total += w;
        acc.x += w * x.x;
        acc.y += w * x.y;
        acc.z += w * x.z;
        acc.w += w * x.w;
    }
    const float inv = total == 0.f ? 0.f : 1.0f / total;
    uint2 out = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2*>(p.o + ((long long)b * Lq + token) * p.ldo + h * 128 + lane * 4) = out;
    if (p.lse && lane == 0)
        p.lse[((long long)b * p.heads + h) * Lq + token] = total == 0.f ? -INFINITY : (m + log2f(total)) * 0.6931471805599453f;
}

cudaError_t init_attention_list_attributes() {
    cudaError_t e = cudaFuncSetAttribute(attn_list_kernel<alist::BLOCKS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         alist::SMEM_BYTES);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_list_kernel<alist::PAGES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 alist::SMEM_BYTES);
    return e;
}

namespace {

// Splits of each list: the number that takes the least time in tile steps.  A
// unit costs its tiles plus about three steps of filling and draining; a split
// one also writes its fp32 rows, and the join reads them all again.
int list_splits(long long per, int max_tiles, int rows) {
    const int streams = 2 * alist::PLAN_SMS;
    if (per >= 8 * streams) return 1;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= 64 && s <= max_tiles; ++s) {
        const long long waves = (per * s + streams - 1) / streams;
        const double share = rows / 128.0;
        const double cost = (double)waves * ((max_tiles + s - 1) / s + 3 + (s > 1 ? share : 0)) +
                            (s > 1 ? 4 + 0.013 * share * per * s : 0);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

long long list_workspace(long long units, int rows, int splits) {
    return splits == 1 ? 0 : units * splits * rows * 129ll * 4;
}

template <alist::Mode MODE>
cudaError_t launch_list(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, ListParams& p, void* ws,
                        const LaunchCtx& ctx) {
    const long long per = (long long)p.nqb * p.heads * p.B;
    p.units = (int)(per * p.splits);
    if (p.splits > 1) {
        p.part_o = reinterpret_cast<float*>(ws);
        p.part_lse = p.part_o + (long long)p.units * p.rows * 128;
    }
    p.scale_log2 = 1.4426950408889634f / sqrtf(128.0f);
    p.wc.err = ctx.err;
    p.wc.limit_ns = ctx.wait_limit_ns;
    const int ctas = (p.units + 1) / 2;
    attn_list_kernel<MODE><<<ctas < ctx.num_sms ? ctas : ctx.num_sms, alist::THREADS, alist::SMEM_BYTES, ctx.stream>>>(tq, tk, tv, p);
    if (ctx.launches) ++*ctx.launches;
    if (p.splits > 1) {
        list_join_kernel<MODE><<<(unsigned)((per * p.rows + 7) / 8), 256, 0, ctx.stream>>>(p);
        if (ctx.launches) ++*ctx.launches;
    }
    return cudaGetLastError();
}

int log2_of(int v) {
    int n = 0;
    while ((1 << n) < v) ++n;
    return n;
}

bool blocks_plan(int B, int heads, const BlockGrid& g, int topk, ListParams* p) {
    p->B = B;
    p->heads = heads;
    p->g = g;
    p->nqb = g.q_blocks();
    p->nkb = g.k_blocks();
    p->rows = g.q_volume();
    p->topk = topk;
    p->log_group = log2_of(g.k_volume());
    p->E = 128 >> p->log_group;
    const long long per = (long long)p->nqb * heads * B;
    p->splits = list_splits(per, (topk + p->E - 1) / p->E, p->rows);
    return per * p->splits < (1ll << 31) - 1024;
}

bool pages_plan(int B, int heads, int T, int max_pages, int page_size, ListParams* p) {
    p->B = B;
    p->heads = heads;
    p->T = T;
    p->nqb = (T + 127) / 128;
    p->rows = T < 128 ? T : 128;
    p->max_pages = max_pages;
    p->log_group = log2_of(page_size);
    p->E = 128 >> p->log_group;
    const long long per = (long long)p->nqb * heads * B;
    p->splits = list_splits(per, (max_pages + p->E - 1) / p->E, p->rows);
    return per * p->splits < (1ll << 31) - 1024;
}

}  // namespace

long long attention_blocks_workspace(int B, int heads, const BlockGrid& g, int topk) {
    ListParams p{};
    if (!blocks_plan(B, heads, g, topk, &p)) return -1;
    return list_workspace((long long)p.nqb * heads * B, p.rows, p.splits);
}

long long attention_paged_workspace(int B, int heads, int T, int max_pages, int page_size) {
    ListParams p{};
    if (!pages_plan(B, heads, T, max_pages, page_size, &p)) return -1;
    return list_workspace((long long)p.nqb * heads * B, p.rows, p.splits);
}

cudaError_t launch_attention_blocks(const void* q, long long ldq, const void* k, long long ldk, const void* v,
                                    long long ldv, void* o, long long ldo, int B, int heads, const BlockGrid& g,
                                    const int* blocks, const int* counts, int topk, float* lse, void* ws,
                                    const LaunchCtx& ctx) {
    ListParams p{};
    if (!blocks_plan(B, heads, g, topk, &p)) return cudaErrorInvalidValue;
    p.blocks = blocks;
    p.counts = counts;
    p.o = reinterpret_cast<__nv_bfloat16*>(o);
    p.ldo = ldo;
    p.lse = lse;
    auto map = [&](CUtensorMap* m, const void* ptr, long long ld, const int (&n)[3], const int (&box)[3]) {
        const uint64_t W = n[2], H = n[1], F = n[0];
        const uint64_t dims[5] = {(uint64_t)heads * 128, W, H, F, (uint64_t)B};
        const uint64_t strides[4] = {(uint64_t)ld, W * ld, W * H * ld, W * H * F * ld};
        return make_tmap_5d(m, ptr, dims, strides, 64, box[2], box[1], box[0]);
    };
    CUtensorMap tq, tk, tv;
    if (!map(&tq, q, ldq, g.q, g.qb) || !map(&tk, k, ldk, g.k, g.kb) || !map(&tv, v, ldv, g.k, g.kb))
        return cudaErrorInvalidValue;
    return launch_list<alist::BLOCKS>(tq, tk, tv, p, ws, ctx);
}

cudaError_t launch_attention_paged(const void* q, long long ldq, const KvPages& c, const int* lens, void* o,
                                   long long ldo, int B, int heads, int T, float* lse, void* ws, const LaunchCtx& ctx) {
    ListParams p{};
    if (!pages_plan(B, heads, T, c.max_pages, c.page_size, &p)) return cudaErrorInvalidValue;
    p.table = c.table;
    p.table_ld = c.table_ld;
    p.num_pages = c.num_pages;
    p.lens = lens;
    p.o = reinterpret_cast<__nv_bfloat16*>(o);
    p.ldo = ldo;
    p.lse = lse;
    const uint64_t width = (uint64_t)heads * 128;
    CUtensorMap tq, tk, tv;
    if (!make_tmap_3d(&tq, q, width, T, B, ldq, (uint64_t)ldq * T, 64, 128) ||
        !make_tmap_3d(&tk, c.k, width, c.page_size, c.num_pages, c.token_stride, c.page_stride, 64, c.page_size) ||
        !make_tmap_3d(&tv, c.v, width, c.page_size, c.num_pages, c.token_stride, c.page_stride, 64, c.page_size))
        return cudaErrorInvalidValue;
    return launch_list<alist::PAGES>(tq, tk, tv, p, ws, ctx);
}

}  // namespace wan
