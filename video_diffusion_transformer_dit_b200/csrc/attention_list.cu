// Attention over listed parts of the sequence, head_dim 128, bf16 operands,
// fp32 softmax:
//   blocks  each query block (a box of up to 128 tokens of the query grid)
//           attends to the key blocks listed for it (boxes of 16..128 tokens);
//   pages   the T new tokens of each sequence attend to the sequence's cached
//           keys and values, which lie in pages of 16..128 tokens.
// One or two new tokens have a kernel of their own, paged_rows_kernel, on the same ranges
// of pages.  Otherwise both are the same loop: a list of token groups, gathered by TMA into tiles of
// 64 keys (a block or page of 128 tokens is two groups), softmax with a running
// maximum and sum, O += P V per tile.
//
// A work unit is one query tile (up to 128 rows of one head and sample) and one
// split of its list.  A CTA (one per SM) carries two units side by side
// (streams t = 0, 1), each with its own Q tile, so one stream's exponentials
// overlap the other's MMAs although the two read different keys.  A stream has
// 256 columns of tensor memory: O_t (128) and two S buffers of 64 columns, each
// overwritten by its P (bf16, 32 columns).  In step k of its unit a stream issues
// S(k) = Q K_k^T into the one buffer and O += P(k-1) V_(k-1) from the other, so
// the softmax finds S(k) finished when it is done with tile k - 1.  (The first
// version had one 128-key S per stream, softmax and MMAs of a stream in turns, and
// one producer and one issuer for both streams: 2.0 ms at the 480p size below.
// 128-key tiles with a producer and an issuer per stream have not been measured.)
// The streams share nothing but the SM: each has its producer,
// its issuer, its softmax warps and its ring of five 16 KB slots for K and V tiles
// in the order K(k), V(k - 1).  Stream t walks units blockIdx.x * 2 + t,
// + 2 * gridDim.x, ...
//
// Every barrier that advances once per tile exists once per S buffer: a waiting
// warp is then at most one phase behind (S(k) is issued after P.V of tile k - 2,
// which waits for the P of tile k - 2), so the phase's parity names it.
//
// Warps (registers per thread as in the dense kernel):
//   0, 2   TMA producer of stream 0 / 1 and the 64-bit mask of each tile's keys (one
//          producer for both streams is the bottleneck: gathering a tile takes it
//          about as long as the tile's MMAs, 2.6 ms);
//   1, 3   MMA issuer of stream 0 / 1 (1 owns the tensor memory); it also zeroes the
//          V rows of a tile past the sequence's end inside a page before its P.V;
//   4..11  softmax of stream 0 / 1, one query row per thread; warps without a
//          row only keep the barriers' counts.
// Where there are too few query tiles to fill the GPU, lists are split.  Blocks:
// each list into `splits` parts.  Pages: sequences differ in length, so the tiles
// of all sequences, one after the other, are cut into `splits` even ranges, and a
// unit is one range for one head and query tile; it may hold the end of one
// sequence, whole ones and the beginning of another.  A part of a list writes its
// normalised fp32 rows and their log-sum-exp, and list_join_kernel joins them.
//
// Measured (12 heads, 32760 tokens of a 480p clip; Tflop/s of the tiles computed):
//   blocks, 336 query blocks of 128 x 78 of 624 key blocks of 64: 1.13-1.2 ms cold, 1.29-1.31
//     in a long run, where the power limit holds the clock at 1.7 GHz; 1.03-1.15 Pflop/s,
//     tensor pipe 57 %.  A third of the rows and keys are padding of blocks at the grid's
//     edges.  What bounds it: S = Q K^T with 64 keys reads both operands from shared
//     memory, 48 clocks where the MMA alone takes 32, and every 128 x 64 tile brings its
//     own K and V, 10.4 GB, 8 TB/s, over the L2.
//   pages, 1560 new tokens on 32760: 363 us with 9 ranges of 156 units, 0.86 Pflop/s.
// Tried on the 480p blocks and slower: Q in tensor memory and one query tile per CTA with
// two threads per row (1.4 ms); two warpgroups on alternate tiles of one query tile (1.36
// in a long run); skipping the MMA steps behind a tile's last key (blocks 1 % faster,
// pages 2 % slower).
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace wan {

namespace alist {
constexpr int KEYS = 64;                   // keys per tile
constexpr int Q_BYTES = 128 * 128 * 2;     // 128 rows x 128 columns: two 64-column swizzled halves
constexpr int Q_HALF = 128 * 128;
constexpr int SLOT_BYTES = KEYS * 128 * 2; // a K or V tile: two 64-column halves
constexpr int KV_HALF = KEYS * 128;
constexpr int SLOTS = 5;                   // per stream
constexpr int MASKS = 16;                  // key masks per stream (tiles in flight: at most 6)
constexpr int SQ = 0;
constexpr int SKV = SQ + 2 * Q_BYTES;
constexpr int SMASK = SKV + 2 * SLOTS * SLOT_BYTES;
constexpr int SBAR = SMASK + 2 * MASKS * 8;
constexpr int SSTART = SBAR + 320;         // pages: first tile of each sequence
constexpr int MAX_SEQS = 256;              // sequences per launch (pages)
constexpr int ROWS_MOST = 2;               // new tokens per sequence that paged_rows_kernel takes
constexpr int SMEM_BYTES = SSTART + (MAX_SEQS + 1) * 4 + 1024;
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
    int E, log_group;       // token groups per tile, log2 of tokens per group (at most 64)
    int log_sub;            // log2 of groups per block or page (1 for 128 tokens)
    // blocks
    BlockGrid g;
    int sub[3], step[3];    // box of one group; offset of a block's second group
    int nk1, nk2;           // key blocks along rows and columns
    FastDiv by_nk2, by_nk1;
    const int* blocks;
    const int* counts;
    int topk, nkb;
    // pages
    const int* table;
    long long table_ld;
    const int* lens;
    int max_pages, num_pages, T;
    int row_warps;          // warps per CTA of paged_rows_kernel
    __nv_bfloat16* o;
    long long ldo;
    float* lse;             // [B, heads, query tokens] or null
    float* part_o;          // [unit][rows][128] fp32 (splits > 1)
    float* part_lse;        // [unit][rows], log2 units
    float scale_log2;
    WaitCtl wc;
};

// One list or part of one: its head, sample, query tile and tiles [j0, j0 + n).
struct ListUnit {
    int b, h, qt, j0, n;
    int length;             // groups in the list (blocks) or tokens in the cache (pages)
    long long part;         // place of its partial rows, -1: the whole list, written to the output
    bool dirty;             // pages: the last tile ends inside a page
};

// Tiles of sequence b of a paged cache, and its tokens.
__device__ __forceinline__ int page_tokens(const ListParams& p, int b) {
    return min(max(__ldg(p.lens + b), 0), p.max_pages << (p.log_group + p.log_sub));
}
__device__ __forceinline__ uint32_t page_tiles(int tokens) { return ((uint32_t)tokens + alist::KEYS - 1) / alist::KEYS; }

// Ranges in use: none without a tile (but for the one that all empty sequences fall to).
__device__ __forceinline__ uint32_t page_ranges(const ListParams& p, uint32_t total) {
    return min((uint32_t)p.splits, max(total, 1u));
}

// What one stream works through: next() takes the next list (false: none left).
// A list without keys comes with n = 0 (blocks also an empty part of a list).  WIDTH
// streams per CTA.
template <alist::Mode MODE, int WIDTH = 2>
struct ListWalk {
    ListUnit x;
    int u, b;                  // unit; pages: next sequence of the range
    uint32_t lo, hi;           // pages: the unit's range of tiles
    const uint32_t* start;     // pages: first tile of each sequence, [B + 1]
    __device__ __forceinline__ ListWalk(int t, const uint32_t* starts)
        : u(blockIdx.x * WIDTH + t - WIDTH * gridDim.x), b(0x7fffffff), lo(0), hi(0), start(starts) {}

    __device__ __forceinline__ bool next(const ListParams& p) {
        if constexpr (MODE == alist::BLOCKS) {
            u += WIDTH * gridDim.x;
            if (u >= p.units) return false;
            // splits slowest: CTAs that run together read the same tokens of several heads
            const int per = p.nqb * p.heads * p.B;
            const int s = u / per;
            int r = u - s * per;
            x.qt = r % p.nqb;
            r /= p.nqb;
            x.h = r % p.heads;
            x.b = r / p.heads;
            const int c = __ldg(p.counts + ((long long)x.b * p.heads + x.h) * p.nqb + x.qt);
            x.length = min(max(c, 0), p.topk) << p.log_sub;
            const int tiles = (x.length + p.E - 1) / p.E;
            x.j0 = (int)((long long)tiles * s / p.splits);
            x.n = (int)((long long)tiles * (s + 1) / p.splits) - x.j0;
            x.part = p.splits > 1 ? u : -1;
            x.dirty = false;
            return true;
        } else while (true) {
            if (b < p.B && (start[b] < hi || (start[b] == hi && hi == start[p.B]))) {
                const uint32_t first = start[b], end = start[b + 1];
                x.b = b++;
                const uint32_t s0 = max(first, lo), s1 = min(end, hi);
                if (end > first && s1 <= s0) continue;
                x.length = page_tokens(p, x.b);
                x.j0 = (int)(s0 - first);
                x.n = end > first ? (int)(s1 - s0) : 0;
                x.part = end > first && (s0 != first || s1 != end) ? u * 2ll + (s0 > lo) : -1;
                x.dirty = s1 == end && (x.length & ((1 << p.log_group) - 1)) != 0;
                return true;
            }
            u += WIDTH * gridDim.x;
            if (u >= p.units) return false;
            const int inner = p.nqb * p.heads;
            const uint32_t r = (uint32_t)(u / inner);
            const int i = u - (int)r * inner;
            x.qt = i % p.nqb;
            x.h = i / p.nqb;
            const uint32_t total = start[p.B], ranges = page_ranges(p, total);
            b = p.B;
            if (r >= ranges) continue;
            lo = (uint32_t)((unsigned long long)total * r / ranges);
            hi = (uint32_t)((unsigned long long)total * (r + 1) / ranges);
            int b0 = 0, b1 = p.B;  // first sequence with tiles at or past lo (or none, at lo)
            while (b0 < b1) {
                const int m = (b0 + b1) >> 1;
                if (start[m + 1] > lo || start[m] >= lo) b1 = m;
                else b0 = m + 1;
            }
            b = b0;
        }
    }
    // the next list that has tiles
    __device__ __forceinline__ bool next_tiles(const ListParams& p) {
        do {
            if (!next(p)) return false;
            // read by every lane alike, but known to the compiler as warp-uniform only from
            // a broadcast: ring slots and descriptors that follow from it stay in uniform registers
            x.n = __shfl_sync(0xffffffffu, x.n, 0);
        } while (x.n == 0);
        return true;
    }
};

// First tile of each sequence (one warp).
__device__ __forceinline__ void page_starts(const ListParams& p, uint32_t* starts, int lane) {
    uint32_t before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        uint32_t n = b0 + lane < p.B ? page_tiles(page_tokens(p, b0 + lane)) : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t m = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += m;
        }
        if (b0 + lane < p.B) starts[b0 + lane + 1] = before + n;
        before += __shfl_sync(0xffffffffu, n, 31);
    }
    if (lane == 0) starts[0] = 0;
}

// Query token of row r of query tile qt, -1 where the tile has no such row.
template <alist::Mode MODE>
__device__ __forceinline__ int list_token(const ListParams& p, int qt, int r) {
    if (MODE == alist::PAGES) return qt * 128 + r < p.T ? qt * 128 + r : -1;
    const int nj = p.g.nq(2), ni = p.g.nq(1);
    const int f = (qt / nj / ni) * p.g.qb[0] + r / (p.g.qb[2] * p.g.qb[1]);
    const int i = (qt / nj % ni) * p.g.qb[1] + r / p.g.qb[2] % p.g.qb[1];
    const int j = (qt % nj) * p.g.qb[2] + r % p.g.qb[2];
    return r < p.rows && f < p.g.q[0] && i < p.g.q[1] && j < p.g.q[2] ? (f * p.g.q[1] + i) * p.g.q[2] + j : -1;
}

// Origin of a token group; an out-of-range sample or page where there is none
// (TMA fills zeros).
struct ListGroup {
    int f, i, j, b;  // blocks: token coordinates and sample; pages: first place, row in the page, -, page
    bool ok;
};

// mbar_spin by a whole warp: one probe and one vote where the phase is complete
// (the usual case), no divergence.
__device__ __forceinline__ bool warp_spin(uint64_t* bar, uint32_t parity, volatile int* abort, const WaitCtl& wc) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t n = 1;; ++n) {
        if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
        if ((n & 63) == 0 || wc.limit_ns == 0) {
            const bool late = wc.limit_ns == 0 || global_ns() - t0 > wc.limit_ns;
            if (__any_sync(0xffffffffu, late || *abort)) {
                if (!*abort && wc.err) atomicExch(wc.err, ERR_TIMEOUT);
                *abort = 1;
                __syncwarp();
                return false;
            }
        }
    }
}

template <alist::Mode MODE>
__global__ void __launch_bounds__(alist::THREADS, 1)
    attn_list_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ListParams p) {
    using namespace alist;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint2* masks = reinterpret_cast<uint2*>(smem + SMASK);  // [2][MASKS]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SBAR);
    uint64_t* q_full = bars;                 // [2]
    uint64_t* q_empty = q_full + 2;          // [2] the unit's last S has read Q
    uint64_t* kv_full = q_empty + 2;         // [2][SLOTS]
    uint64_t* kv_empty = kv_full + 2 * SLOTS;  // [2][SLOTS]
    uint64_t* s_full = kv_empty + 2 * SLOTS; // [2][2] stream, S buffer
    uint64_t* p_full = s_full + 4;           // [2][2] P stored over S
    uint64_t* pv_done = p_full + 4;          // [2][2] P.V of the buffer's tile has landed
    uint64_t* drain = pv_done + 4;           // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint32_t* starts = reinterpret_cast<uint32_t*>(smem + SSTART);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full + t, 1);
            mbar_init(q_empty + t, 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(s_full + 2 * t + i, 1);
                mbar_init(p_full + 2 * t + i, 4);
                mbar_init(pv_done + 2 * t + i, 1);
            }
        }
        for (int s = 0; s < 2 * SLOTS; ++s) {
            mbar_init(kv_full + s, 1);
            mbar_init(kv_empty + s, 1);
        }
        mbar_init(drain, 1);
        mbar_init(drain + 1, 1);
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
    if (MODE == PAGES && warp == 2) page_starts(p, starts, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    // every CTA is resident: the join may take the SMs that are done, and wait
    if (p.splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // producer: slots with a load issued and the phase it completes, phase of the
    // last Q load; issuer: whether any MMA went out (both drained after an abort)
    uint32_t armed = 0, par = 0;
    int qpar = -1;
    bool issued = false;

    if (warp < 4) {
        regs_dealloc<REGS_CONTROL>();
        const int t = warp >> 1;
        uint8_t* ring = smem + SKV + t * SLOTS * SLOT_BYTES;
        uint64_t* full = kv_full + t * SLOTS;
        uint64_t* empty = kv_empty + t * SLOTS;
        if ((warp & 1) == 0) {
            // ---------------- producer of stream t ----------------
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                return warp_spin(bar, parity, abort_flag, p.wc);
            };
            const int group = 1 << p.log_group;
            // place of the lane's two key columns inside their group
            int off[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = (c * 32 + lane) & (group - 1);
                off[c] = r;
                if (MODE == BLOCKS) {
                    const int dj = r % p.sub[2], di = (r / p.sub[2]) % p.sub[1], df = r / (p.sub[2] * p.sub[1]);
                    off[c] = df | di << 8 | dj << 16;
                }
            }
            // lane e: the list's entry for group e of tile j (bounded by the list's room:
            // the load does not wait for its length), and the group it names
            auto fetch = [&](const ListUnit& x, int j) -> int {
                const int idx = (j * p.E + lane) >> p.log_sub;
                if (lane >= p.E || idx >= (MODE == BLOCKS ? p.topk : p.max_pages)) return -1;
                return MODE == BLOCKS
                           ? __ldg(p.blocks + (((long long)x.b * p.heads + x.h) * p.nqb + x.qt) * p.topk + idx)
                           : __ldg(p.table + (long long)x.b * p.table_ld + idx);
            };
            auto group_of = [&](const ListUnit& x, int j, int id) -> ListGroup {
                ListGroup o{0, 0, 0, MODE == BLOCKS ? p.B : p.num_pages, false};
                const int idx = j * p.E + lane;
                if (MODE == BLOCKS) {
                    if (idx >= x.length || id < 0 || id >= p.nkb) return o;
                    const int r = p.by_nk2(id), f = p.by_nk1(r);
                    const int second = idx & ((1 << p.log_sub) - 1);
                    o.j = (id - r * p.nk2) * p.g.kb[2] + second * p.step[2];
                    o.i = (r - f * p.nk1) * p.g.kb[1] + second * p.step[1];
                    o.f = f * p.g.kb[0] + second * p.step[0];
                    o.b = x.b;
                } else {
                    if ((idx << p.log_group) >= x.length || id < 0 || id >= p.num_pages) return o;
                    o.b = id;
                    o.f = idx << p.log_group;
                    o.i = (idx & ((1 << p.log_sub) - 1)) << p.log_group;
                }
                o.ok = true;
                return o;
            };
            auto write_mask = [&](const ListUnit& x, const ListGroup& o, uint2* dst) {
                uint32_t w[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
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
                if (lane == 0) *dst = make_uint2(w[0], w[1]);
                // before the elected lane's arrival on the tile's barrier, which publishes the mask:
                // votes and shuffles between the two order no memory
                __syncwarp();
            };
            // the tile's groups into a slot: coordinates broadcast, one lane issues all copies from
            // uniform registers (a copy per lane is issued lane by lane, three times as slow)
            auto gather = [&](auto groups, const CUtensorMap* tm, uint8_t* dst, uint64_t* bar, int h0, const ListGroup& o) {
                constexpr int E = decltype(groups)::value;
                int f[E], i[E], j[E], b[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    i[e] = __shfl_sync(0xffffffffu, o.i, e);
                    b[e] = __shfl_sync(0xffffffffu, o.b, e);
                    if (MODE == BLOCKS) {
                        f[e] = __shfl_sync(0xffffffffu, o.f, e);
                        j[e] = __shfl_sync(0xffffffffu, o.j, e);
                    }
                }
                if (elect_one()) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint8_t* to = dst + half * KV_HALF + e * (KEYS / E) * 128;
                            if (MODE == BLOCKS)
                                tma_load_5d(to, tm, bar, h0 + half * 64, j[e], i[e], f[e], b[e]);
                            else
                                tma_load_3d(to, tm, bar, h0 + half * 64, i[e], b[e]);
                        }
                }
                __syncwarp();
            };
            int c = 0;  // loads so far
            auto load = [&](const CUtensorMap* tm, const ListUnit& x, const ListGroup& o) -> bool {
                const int slot = c % SLOTS;
                const uint32_t phase = (c / SLOTS) & 1;
                ++c;
                if (!wait(empty + slot, phase ^ 1)) return false;
                if (elect_one()) mbar_expect_tx(full + slot, SLOT_BYTES);
                __syncwarp();
                uint8_t* dst = ring + slot * SLOT_BYTES;
                if (p.E == 1)
                    gather(std::integral_constant<int, 1>{}, tm, dst, full + slot, x.h * 128, o);
                else if (p.E == 2)
                    gather(std::integral_constant<int, 2>{}, tm, dst, full + slot, x.h * 128, o);
                else
                    gather(std::integral_constant<int, 4>{}, tm, dst, full + slot, x.h * 128, o);
                armed |= 1u << slot;
                par = (par & ~(1u << slot)) | phase << slot;
                return true;
            };
            ListWalk<MODE> w(t, starts);
            ListGroup last;  // the previous tile's groups: its V goes one step after its K
            int tiles = 0, unit = 0;
            bool ok = true, more = w.next_tiles(p);
            int ahead = more ? fetch(w.x, w.x.j0) : -1;  // entries of the next tile, loaded a step ahead
            while (ok && more) {
                const ListUnit x = w.x;
                if (!wait(q_empty + t, (unit & 1) ^ 1)) break;
                if (elect_one()) {
                    uint8_t* dst = smem + SQ + t * Q_BYTES;
                    const int h0 = x.h * 128;
                    if (MODE == BLOCKS) {
                        const int nj = p.g.nq(2), ni = p.g.nq(1);
                        const int j = (x.qt % nj) * p.g.qb[2], i = (x.qt / nj % ni) * p.g.qb[1], f = (x.qt / nj / ni) * p.g.qb[0];
                        mbar_expect_tx(q_full + t, p.rows * 256);
                        tma_load_5d(dst, &tmQ, q_full + t, h0, j, i, f, x.b);
                        tma_load_5d(dst + Q_HALF, &tmQ, q_full + t, h0 + 64, j, i, f, x.b);
                    } else {
                        mbar_expect_tx(q_full + t, Q_BYTES);
                        tma_load_3d(dst, &tmQ, q_full + t, h0, x.qt * 128, x.b);
                        tma_load_3d(dst + Q_HALF, &tmQ, q_full + t, h0 + 64, x.qt * 128, x.b);
                    }
                }
                __syncwarp();
                qpar = unit & 1;
                ++unit;
                for (int k = 0; ok && k <= x.n; ++k) {
                    const ListGroup prev = last;
                    if (k < x.n) {
                        last = group_of(x, x.j0 + k, ahead);
                        if (k + 1 < x.n) {
                            ahead = fetch(x, x.j0 + k + 1);
                        } else {
                            more = w.next_tiles(p);
                            if (more) ahead = fetch(w.x, w.x.j0);
                        }
                        write_mask(x, last, masks + t * MASKS + (tiles & (MASKS - 1)));
                        ++tiles;
                        ok = load(&tmK, x, last);
                    }
                    if (ok && k > 0) ok = load(&tmV, x, prev);
                }
            }
        } else {
            // ---------------- MMA issuer of stream t ----------------
            // the whole warp runs the loop; one elected lane issues
            constexpr uint32_t ID_QK = idesc_bf16(128, KEYS, false);
            constexpr uint32_t ID_PV = idesc_bf16(128, 128, true);
            const uint64_t dq = sdesc_kmajor_sw128(smem_u32(smem + SQ + t * Q_BYTES));
            const uint64_t dk = sdesc_kmajor_sw128(smem_u32(ring));
            const uint64_t dv = sdesc_mnmajor_sw128(smem_u32(ring), KV_HALF);
            const uint32_t ts = tmem + t * 128, to = tmem + 256 + t * 128;
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                return warp_spin(bar, parity, abort_flag, p.wc);
            };
            ListWalk<MODE> w(t, starts);
            int c = 0, tiles = 0, unit = 0;
            bool ok = true;
            while (ok && w.next_tiles(p)) {
                const int n = w.x.n;
                if (!wait(q_full + t, unit & 1)) break;
                ++unit;
                for (int k = 0; k <= n; ++k) {
                    const int at = tiles;  // tile k, counted over the stream's units
                    if (k < n) {
                        // S(k): its buffer held P(k - 2), whose P.V went out two steps ago
                        const int slot = c % SLOTS;
                        const uint32_t phase = (c / SLOTS) & 1;
                        ++c;
                        if (!wait(full + slot, phase)) { ok = false; break; }
                        tc_fence_after();
                        const uint64_t b = dk + (uint64_t)((slot * SLOT_BYTES) >> 4);
                        const uint32_t d = ts + (at & 1) * KEYS;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                umma_bf16_ss(d, dq + (((kk >> 2) * Q_HALF + (kk & 3) * 32) >> 4),
                                             b + (((kk >> 2) * KV_HALF + (kk & 3) * 32) >> 4), ID_QK, kk != 0);
                            umma_commit(s_full + 2 * t + (at & 1));
                            umma_commit(empty + slot);
                            if (k == n - 1) umma_commit(q_empty + t);
                        }
                        __syncwarp();
                        issued = true;
                        ++tiles;
                    }
                    if (k > 0) {
                        // O += P(k - 1) V(k - 1)
                        const int slot = c % SLOTS;
                        const uint32_t phase = (c / SLOTS) & 1;
                        ++c;
                        const int prev = at - 1;
                        if (!wait(full + slot, phase)) { ok = false; break; }
                        if (MODE == PAGES && k == n && w.x.dirty) {
                            // rows past the sequence hold foreign memory: 0 * NaN would reach O
                            const int valid = w.x.length - (w.x.j0 + n - 1) * KEYS;  // 1..63
                            const uint32_t base = smem_u32(ring + slot * SLOT_BYTES);
                            for (int i = valid * 8 + lane; i < KEYS * 8; i += 32) {
                                st_shared_v4(base + i * 16, 0, 0, 0, 0);
                                st_shared_v4(base + KV_HALF + i * 16, 0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        if (!wait(p_full + 2 * t + (prev & 1), (prev >> 1) & 1)) { ok = false; break; }
                        tc_fence_after();
                        const uint64_t b = dv + (uint64_t)((slot * SLOT_BYTES) >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < KEYS / 16; ++kk)
                                umma_bf16_ts(to, ts + (prev & 1) * KEYS + kk * 8, b + ((kk * 2048) >> 4), ID_PV,
                                             !(k == 1 && kk == 0));
                            umma_commit(empty + slot);
                            umma_commit(pv_done + 2 * t + (prev & 1));
                        }
                        __syncwarp();
                    }
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
        const uint32_t TS0 = tmem + t * 128 + lane_off;  // the S (and P) buffers
        const uint32_t TO = tmem + 256 + t * 128 + lane_off;
        bool ok = true;
        int g = 0;  // tiles so far
        ListWalk<MODE> w(t, starts);
        while (w.next(p)) {
            const int n = w.x.n;
            const int token = list_token<MODE>(p, w.x.qt, r);
            const bool active = __any_sync(0xffffffffu, token >= 0);
            float m_run = -INFINITY, l_run = 0.0f;
            for (int j = 0; j < n; ++j, ++g) {
                const int buf = g & 1;
                const uint32_t TS = TS0 + buf * KEYS;
                // all tcgen05.ld/st below are warp-collective: the warp's decisions stay uniform
                if (!__all_sync(0xffffffffu, mbar_wait(s_full + 2 * t + buf, (g >> 1) & 1, abort_flag, p.wc))) { ok = false; break; }
                tc_fence_after();
                if (!active) {  // no row here: the S columns stay as they are, nothing reads their product
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 2 * t + buf);
                    continue;
                }
                uint32_t sv[2][32];
                tmem_ld32(TS, sv[0]);
                tmem_ld32(TS + 32, sv[1]);
                const uint2 mk = masks[t * MASKS + (g & (MASKS - 1))];
                tmem_ld_wait(sv[0]);
                tmem_ld_wait(sv[1]);
                if ((mk.x & mk.y) != 0xffffffffu) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t w = c ? mk.y : mk.x;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(w >> i & 1)) sv[c][i] = __float_as_uint(-INFINITY);
                    }
                }
                // row maximum: four independent 3-input max chains
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t* v = &sv[q >> 1][(q & 1) * 16];
                    float a = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
#pragma unroll
                    for (int i = 2; i < 16; i += 2) a = max3f(a, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                    mx[q] = a;
                }
                const float m_tile = fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
                const float m_new = fmaxf(m_run, m_tile);
                const bool rescale = m_new > m_run + RESCALE_THRESHOLD;
                const float m_use = rescale ? m_new : m_run;
                const float m_sub = m_use == -INFINITY ? 0.0f : m_use;  // every key so far masked: all exponentials are 0
                const float alpha = rescale ? ex2_approx(m_run - m_use) : 1.0f;  // 0 on the first tile
                if (j > 0 && __any_sync(0xffffffffu, rescale)) {
                    // O_t is scaled between the P.V of the previous tile and this tile's
                    if (!__all_sync(0xffffffffu, mbar_wait(pv_done + 2 * t + ((g - 1) & 1), ((g - 1) >> 1) & 1, abort_flag, p.wc))) { ok = false; break; }
                    tc_fence_after();
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
                // tensor core's operand type: half a step is 2^-8 of each) over their S columns
                uint64_t ps2[2] = {0ull, 0ull};
                const uint64_t scale2 = f2pack(p.scale_log2, p.scale_log2);
                const uint64_t negm2 = f2pack(-m_sub, -m_sub);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
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
                if (lane == 0) mbar_arrive(p_full + 2 * t + buf);
            }
            if (!ok) break;
            // the unit's output: O_t / l once its last P.V has landed (zero rows where no key was left)
            if (n > 0) {
                if (!__all_sync(0xffffffffu, mbar_wait(pv_done + 2 * t + ((g - 1) & 1), ((g - 1) >> 1) & 1, abort_flag, p.wc))) { ok = false; break; }
                tc_fence_after();
            }
            if (!active) continue;
            const bool none = l_run == 0.0f;
            const float inv = none ? 0.0f : 1.0f / l_run;
            const float lse2 = none ? -INFINITY : m_run + log2f(l_run);
            const bool direct = w.x.part < 0;
            const int Lq = MODE == BLOCKS ? p.g.q_tokens() : p.T;
            if (token >= 0) {
                if (!direct)
                    p.part_lse[w.x.part * p.rows + r] = lse2;
                else if (p.lse)
                    p.lse[((long long)w.x.b * p.heads + w.x.h) * Lq + token] = lse2 * 0.6931471805599453f;
            }
            __nv_bfloat16* orow = p.o + ((long long)w.x.b * Lq + token) * p.ldo + w.x.h * 128;
            if (n == 0) {  // a list without keys; the join does not read rows whose sum is empty
                if (direct && token >= 0)
                    for (int c = 0; c < 16; ++c) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0, 0, 0, 0);
                continue;
            }
            float* prow = p.part_o + (w.x.part * p.rows + r) * 128;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t ov[32];
                tmem_ld32(TO + c * 32, ov);
                tmem_ld_wait(ov);
#pragma unroll
                for (int i = 0; i < 32; ++i) ov[i] = none ? 0u : ov[i];
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
        if (warp == 0 || warp == 2) {
            const int t = warp >> 1;
            if (lane == 0) {
                if (qpar >= 0) mbar_drain(q_full + t, static_cast<uint32_t>(qpar), 200000000ull);
                for (int s = 0; s < SLOTS; ++s)
                    if (armed & (1u << s)) mbar_drain(kv_full + t * SLOTS + s, (par >> s) & 1, 200000000ull);
            }
        } else if ((warp == 1 || warp == 3) && issued) {
            if (elect_one()) {  // the lane that issued the MMAs
                umma_commit(drain + (warp >> 1));
                mbar_drain(drain + (warp >> 1), 0, 200000000ull);
            }
            __syncwarp();
        }
        __syncthreads();
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// R new tokens per sequence (p.T == R): no product is wide enough for the tensor cores, and
// K and V go through registers once.  A CTA takes one unit (a range of tiles for one
// head) at a time, its warps 16 keys each in turn: a half warp reads a key's 128 columns
// (16 bytes per lane, eight keys in flight), and
//   s_i = sum over 8 columns in fp32 pairs, then over the 16 lanes with the keys
//         dealt out on the way, so that a lane pair ends with one key's score;
//   p   = 2^(s - m) per lane pair, m the warp's running maximum;
//   o  += p_i v_i, p_i fetched from its lanes.
// p stays fp32.  The warps' (m, l, o) meet in shared memory at the unit's end.
//
// Memory bound: one token, 12 heads, 131040 places: 119.8 us cold, 123.2 in a long run (6.6
// TB/s); a copy of as many bytes takes 123.  The tiles take 127.5 and 133.6, as their MMAs
// are 128 rows wide all the same: tensor cores and shared memory draw the power that the
// memory wants, and the clock falls to 1.45 GHz.  4096 places: 10.0 us against 15.1.  Two
// tokens: 134.8 against 135.5 and 14.1 against 18.5; from three on the arithmetic, 13
// instructions per key and row beside the 22 that all rows share, bounds it: 224 us
// against 137.  So R is 1 or 2; 16 warps to an SM (eight keys of K and V in flight per
// lane, 116 and 128 registers), in two CTAs, or in four where there are more lists than
// such units: each list ends with the meeting of its warps (256 sequences of 64 tokens: 34.5
// against 44.1 us, of 130: 52 against 64; one of 4096: 11.9 against 10.1, more parts to join).
// The rule goes by the number of lists alone, as lengths are known on the device only: with
// long lists the two are within 2 %, 300 to 1280 of 2000 to 16380 places 62 to 352 us in two CTAs
// and 63 to 355 in four (two tokens: 66 to 365 and 67 to 365).
template <int R, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) paged_rows_kernel(const __nv_bfloat16* __restrict__ q, long long ldq,
                                                            const __nv_bfloat16* __restrict__ k,
                                                            const __nv_bfloat16* __restrict__ v,
                                                            long long page_stride, long long token_stride,
                                                            const __grid_constant__ ListParams p) {
    using namespace alist;
    __shared__ uint32_t starts[MAX_SEQS + 1];
    __shared__ float warp_m[WARPS][R], warp_l[WARPS][R];
    __shared__ __align__(16) float warp_o[WARPS][R][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) page_starts(p, starts, lane);
    __syncthreads();
    if (p.splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int STEP = WARPS * 16;
    const int sub = lane >> 4, col = (lane & 15) * 8;
    const int log_page = p.log_group + p.log_sub;
    auto pairs = [](const uint4& x, uint64_t (&y)[4]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = f2pack(__uint_as_float(w[c] << 16), __uint_as_float(w[c] & 0xffff0000u));
    };
    auto fetch = [](const __nv_bfloat16* at) {
        uint4 x;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "l"(at));
        return x;
    };
    ListWalk<PAGES, 1> w(0, starts);
    while (w.next(p)) {
        const ListUnit x = w.x;
        uint64_t q2[R][4], acc[R][4];
        float m[R], l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            pairs(__ldg(reinterpret_cast<const uint4*>(q + ((long long)x.b * p.T + r) * ldq + x.h * 128 + col)), q2[r]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                q2[r][c] = mul2(q2[r][c], f2pack(p.scale_log2, p.scale_log2));
                acc[r][c] = 0ull;
            }
            m[r] = -INFINITY;
            l[r] = 0.f;
        }
        const int end = x.n > 0 ? min(x.length, (x.j0 + x.n) * KEYS) : 0;
        const int* table = p.table + (long long)x.b * p.table_ld;
        int k0 = x.j0 * KEYS + warp * 16;
        int page = k0 < end ? __ldg(table + (k0 >> log_page)) : -1;
        for (; k0 < end; k0 += STEP) {
            const int here = page;
            page = k0 + STEP < end ? __ldg(table + ((k0 + STEP) >> log_page)) : -1;
            if (here < 0 || here >= p.num_pages) continue;
            const long long at = here * page_stride + ((k0 & ((1 << log_page) - 1)) + sub) * token_stride + x.h * 128 + col;
            const int left = end - k0 - sub;  // keys 0, 2, 4 ... of this half warp
            uint4 kx[8], vx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) kx[i] = 2 * i < left ? fetch(k + at + 2 * i * token_stride) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) vx[i] = 2 * i < left ? fetch(v + at + 2 * i * token_stride) : make_uint4(0, 0, 0, 0);
            float s[R][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint64_t y[4];
                pairs(kx[i], y);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    uint64_t d = mul2(y[0], q2[r][0]);
#pragma unroll
                    for (int c = 1; c < 4; ++c) d = fma2(y[c], q2[r][c], d);
                    float a, b;
                    f2unpack(d, a, b);
                    s[r][i] = a + b;
                }
            }
            float prob[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                // over the half warp, half of the keys handed over per step
#pragma unroll
                for (int o = 8, n = 4; o >= 2; o >>= 1, n >>= 1) {
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const float keep = lane & o ? s[r][n + i] : s[r][i], give = lane & o ? s[r][i] : s[r][n + i];
                        s[r][i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
                float t = s[r][0] + __shfl_xor_sync(0xffffffffu, s[r][0], 1);
                const int mine = (lane >> 3 & 1) * 4 + (lane >> 2 & 1) * 2 + (lane >> 1 & 1);
                if (2 * mine >= left) t = -INFINITY;
                float top = t;
#pragma unroll
                for (int o = 16; o >= 2; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (top > m[r]) {  // the whole warp alike
                    const float a = ex2_approx(m[r] - top);
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[r][c] = mul2(acc[r][c], f2pack(a, a));
                    l[r] *= a;
                    m[r] = top;
                }
                prob[r] = ex2_approx(t - (m[r] == -INFINITY ? 0.f : m[r]));
                l[r] += prob[r];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint64_t y[4];
                pairs(vx[i], y);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float pi = __shfl_sync(0xffffffffu, prob[r], (lane & 16) | (i >> 2 & 1) * 8 | (i >> 1 & 1) * 4 | (i & 1) * 2);
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[r][c] = fma2(y[c], f2pack(pi, pi), acc[r][c]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
            float y[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) f2unpack(acc[r][c], y[2 * c], y[2 * c + 1]);
#pragma unroll
            for (int c = 0; c < 8; ++c) y[c] += __shfl_xor_sync(0xffffffffu, y[c], 16);
            if (lane < 16) {
                *reinterpret_cast<float4*>(&warp_o[warp][r][col]) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(&warp_o[warp][r][col + 4]) = make_float4(y[4], y[5], y[6], y[7]);
            }
            if (lane == 0) {
                warp_m[warp][r] = m[r];
                warp_l[warp][r] = 0.5f * l[r];  // two lanes had each key
            }
        }
        __syncthreads();
        // p.T is R: with R the loop is unrolled, and two tokens over 131040 places take 136 us for 127
        for (int e = threadIdx.x; e < p.T * 128; e += WARPS * 32) {
            const int r = e >> 7, d = e & 127;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) top = fmaxf(top, warp_m[i][r]);
            float total = 0.f, o = 0.f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                const float f = warp_m[i][r] == -INFINITY ? 0.f : ex2_approx(warp_m[i][r] - top);
                total += f * warp_l[i][r];
                o += f * warp_o[i][r][d];
            }
            const bool none = total == 0.f;
            o *= none ? 0.f : 1.0f / total;
            const float lse2 = none ? -INFINITY : top + log2f(total);
            if (x.part >= 0) {
                p.part_o[(x.part * p.rows + r) * 128 + d] = o;
                if (d == 0) p.part_lse[x.part * p.rows + r] = lse2;
            } else {
                p.o[((long long)x.b * p.T + r) * p.ldo + x.h * 128 + d] = __float2bfloat16(o);
                if (d == 0 && p.lse) p.lse[((long long)x.b * p.heads + x.h) * p.T + r] = lse2 * 0.6931471805599453f;
            }
        }
        __syncthreads();
    }
}

// Joins the parts of one query row's list: O = sum_s w_s O_s, w_s = 2^(lse_s -
// lse); a part without keys has lse -inf and is not read.  A CTA takes JOIN_ROWS
// rows of one query tile, two per warp: it is latency that bounds it (the first
// 32 parts' lse of both rows in one round, then eight parts' rows at a time).  It is
// launched while the attention kernel still runs and waits for it after its set-up.
constexpr int JOIN_ROWS = 16;
template <alist::Mode MODE>
__global__ void __launch_bounds__(256) list_join_kernel(const __grid_constant__ ListParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = p.nqb * p.heads * p.B;
    const int unit = blockIdx.x;
    const int qt = unit % p.nqb, h = unit / p.nqb % p.heads, b = unit / p.nqb / p.heads;
    const int Lq = MODE == alist::BLOCKS ? p.g.q_tokens() : p.T;
    int s0 = 0, s1 = p.splits - 1;
    bool inside = false;  // pages: the first part begins inside its range
    bool parts = true;    // else written whole by its unit
    if (MODE == alist::PAGES) {
        uint32_t first = 0, total = 0, mine = 0;
        for (int i = lane; i < p.B; i += 32) {
            const uint32_t n = page_tiles(page_tokens(p, i));
            total += n;
            if (i < b) first += n;
            if (i == b) mine = n;
        }
        first = __reduce_add_sync(0xffffffffu, first);
        total = __reduce_add_sync(0xffffffffu, total);
        mine = __reduce_add_sync(0xffffffffu, mine);
        // range that holds tile x: the largest r with floor(r total / ranges) <= x
        const uint32_t ranges = page_ranges(p, total);
        auto range_of = [&](uint32_t x) {
            return (int)(((x + 1ull) * ranges + total - 1) / total) - 1;
        };
        if (mine > 0) {
            s0 = range_of(first);
            s1 = range_of(first + mine - 1);
            inside = (uint32_t)((unsigned long long)total * s0 / ranges) < first;
        }
        parts = mine > 0 && s0 != s1;
    }
    auto part = [&](int s) -> long long {
        if (MODE == alist::BLOCKS) return (long long)s * per + unit;
        const long long u = (long long)s * (p.nqb * p.heads) + h * p.nqb + qt;
        return u * 2 + (s == s0 && inside);
    };
    // The parts are written.  Every CTA waits, also one with nothing to join: work
    // behind this kernel in the stream counts on the attention kernel's end.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!parts) return;
    int token[2];
    float l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = blockIdx.y * JOIN_ROWS + warp * 2 + i;
        token[i] = r < p.rows ? list_token<MODE>(p, qt, r) : -1;
        l[i] = token[i] >= 0 && s0 + lane <= s1 ? p.part_lse[part(s0 + lane) * p.rows + r] : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (token[i] < 0) continue;
        const int r = blockIdx.y * JOIN_ROWS + warp * 2 + i;
        // a lane per part for its lse, then all lanes add up the parts' rows
        float m = l[i];
        for (int s = s0 + lane + 32; s <= s1; s += 32) m = fmaxf(m, p.part_lse[part(s) * p.rows + r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float total = 0.f;
        for (int c = s0; c <= s1; c += 32) {
            const float lc = c == s0 ? l[i] : c + lane <= s1 ? p.part_lse[part(c + lane) * p.rows + r] : -INFINITY;
            const float w = lc == -INFINITY ? 0.0f : exp2f(lc - m);
            const int n = min(32, s1 - c + 1);
            for (int k = 0; k < n; k += 8) {
                float4 x[8];
                float wk[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    wk[j] = k + j < n ? __shfl_sync(0xffffffffu, w, (k + j) & 31) : 0.0f;
                    x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (wk[j] != 0.0f)
                        x[j] = *reinterpret_cast<const float4*>(p.part_o + (part(c + k + j) * p.rows + r) * 128 + lane * 4);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    total += wk[j];
                    acc.x += wk[j] * x[j].x;
                    acc.y += wk[j] * x[j].y;
                    acc.z += wk[j] * x[j].z;
                    acc.w += wk[j] * x[j].w;
                }
            }
        }
        const float inv = total == 0.f ? 0.f : 1.0f / total;
        uint2 out = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2*>(p.o + ((long long)b * Lq + token[i]) * p.ldo + h * 128 + lane * 4) = out;
        if (p.lse && lane == 0)
            p.lse[((long long)b * p.heads + h) * Lq + token[i]] =
                total == 0.f ? -INFINITY : (m + log2f(total)) * 0.6931471805599453f;
    }
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

// Splits of each list: the number that takes the least time in tile steps, over the
// waves of two units per SM.  A unit costs its tiles plus five steps of filling and
// draining, a split one another for its fp32 rows, and the join reads them all again.
// With the tiles, in ten shapes (1 to 1560 rows, 30 to 2049 tiles, every number of splits
// up to 49), its choice was within 3 % of the best one, and 5 % in one; a wave more costs 30
// to 50 %.  paged_rows_kernel is planned by the same numbers: in nine shapes of 5 to 40 heads,
// 700 to 131040 places, within 5 % of the best of fourteen tried.  One head alone over 131040
// places is not: 42.8 us with 296 parts, which one warp per row joins, 27.6 with 111.
int list_splits(long long per, long long max_tiles, int rows, int streams = 2 * alist::PLAN_SMS) {
    if (per <= 0 || per >= 8 * streams) return 1;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= 2 * streams / per + 16 && s <= max_tiles; ++s) {
        const long long waves = (per * s + streams - 1) / streams;
        const double share = rows / 128.0;
        const double cost = (double)waves * ((max_tiles + s - 1) / s + 5 + (s > 1 ? share : 0)) +
                            (s > 1 ? 4 + 0.013 * share * per * s : 0);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

long long list_workspace(long long parts, int rows) { return parts * rows * 129ll * 4; }

// The kernel over p's units, launch(), and the join of split lists.
template <alist::Mode MODE, typename Launch>
cudaError_t launch_list(ListParams& p, void* ws, const LaunchCtx& ctx, Launch launch) {
    const long long per = (long long)p.nqb * p.heads * p.B;
    p.units = MODE == alist::BLOCKS ? (int)(per * p.splits) : p.nqb * p.heads * p.splits;
    if (p.splits > 1) {
        p.part_o = reinterpret_cast<float*>(ws);
        p.part_lse = p.part_o + (long long)p.units * (MODE == alist::BLOCKS ? 1 : 2) * p.rows * 128;
    }
    p.scale_log2 = 1.4426950408889634f / sqrtf(128.0f);
    p.wc.err = ctx.err;
    p.wc.limit_ns = ctx.wait_limit_ns;
    launch();
    if (ctx.launches) ++*ctx.launches;
    if (p.splits > 1) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)per, (p.rows + JOIN_ROWS - 1) / JOIN_ROWS);
        cfg.blockDim = dim3(256);
        cfg.stream = ctx.stream;
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, list_join_kernel<MODE>, static_cast<const ListParams&>(p));
        if (e != cudaSuccess) return e;
        if (ctx.launches) ++*ctx.launches;
    }
    return cudaGetLastError();
}

template <alist::Mode MODE>
cudaError_t launch_tiles(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, ListParams& p, void* ws,
                         const LaunchCtx& ctx) {
    return launch_list<MODE>(p, ws, ctx, [&] {
        const int ctas = (p.units + 1) / 2;
        attn_list_kernel<MODE><<<ctas < ctx.num_sms ? ctas : ctx.num_sms, alist::THREADS, alist::SMEM_BYTES, ctx.stream>>>(
            tq, tk, tv, p);
    });
}

template <int R, int WARPS>
cudaError_t launch_rows(const void* q, long long ldq, const KvPages& c, ListParams& p, void* ws, const LaunchCtx& ctx) {
    return launch_list<alist::PAGES>(p, ws, ctx, [&] {
        const int most = 16 / WARPS * ctx.num_sms;  // resident
        paged_rows_kernel<R, WARPS><<<p.units < most ? p.units : most, WARPS * 32, 0, ctx.stream>>>(
            reinterpret_cast<const __nv_bfloat16*>(q), ldq, reinterpret_cast<const __nv_bfloat16*>(c.k),
            reinterpret_cast<const __nv_bfloat16*>(c.v), c.page_stride, c.token_stride, p);
    });
}

int log2_of(int v) {
    int n = 0;
    while ((1 << n) < v) ++n;
    return n;
}

// Token groups of a block or page of `tokens` (16, 32, 64 or 128) tokens.
void list_groups(int tokens, ListParams* p) {
    p->log_sub = tokens > alist::KEYS ? 1 : 0;
    p->log_group = log2_of(tokens) - p->log_sub;
    p->E = alist::KEYS >> p->log_group;
}

bool blocks_plan(int B, int heads, const BlockGrid& g, int topk, ListParams* p) {
    p->B = B;
    p->heads = heads;
    p->g = g;
    p->nqb = g.q_blocks();
    p->nkb = g.k_blocks();
    p->rows = g.q_volume();
    p->topk = topk;
    list_groups(g.k_volume(), p);
    for (int a = 0; a < 3; ++a) {
        p->sub[a] = g.kb[a];
        p->step[a] = 0;
    }
    p->nk1 = g.nk(1);
    p->nk2 = g.nk(2);
    p->by_nk1 = fast_div(p->nk1);
    p->by_nk2 = fast_div(p->nk2);
    if (p->log_sub) {  // two groups of 64: halves of the block's longest axis (a power of two, as its volume is)
        int a = 0;
        for (int i = 1; i < 3; ++i)
            if (g.kb[i] > g.kb[a]) a = i;
        p->sub[a] = p->step[a] = g.kb[a] / 2;
    }
    const long long per = (long long)p->nqb * heads * B;
    p->splits = list_splits(per, ((topk << p->log_sub) + p->E - 1) / p->E, p->rows);
    return per * p->splits < (1ll << 31) - 1024;
}

bool pages_plan(int B, int heads, int T, int max_pages, int page_size, ListParams* p) {
    p->B = B;
    p->heads = heads;
    p->T = T;
    p->nqb = (T + 127) / 128;
    p->rows = T < 128 ? T : 128;
    p->max_pages = max_pages;
    list_groups(page_size, p);
    const long long inner = (long long)p->nqb * heads;
    const long long tiles = ((long long)max_pages << (p->log_sub + p->log_group)) / alist::KEYS + 1;
    p->row_warps = inner * B > 2 * alist::PLAN_SMS ? 4 : 8;
    p->splits = list_splits(inner, tiles * B, p->rows,
                            T > alist::ROWS_MOST ? 2 * alist::PLAN_SMS : 16 / p->row_warps * alist::PLAN_SMS);
    return inner * p->splits < (1ll << 30);
}

}  // namespace

long long attention_blocks_workspace(int B, int heads, const BlockGrid& g, int topk) {
    ListParams p{};
    if (!blocks_plan(B, heads, g, topk, &p)) return -1;
    return p.splits == 1 ? 0 : list_workspace((long long)p.nqb * heads * B * p.splits, p.rows);
}

long long attention_paged_workspace(int B, int heads, int T, int max_pages, int page_size) {
    ListParams p{};
    if (B == 0 || T == 0) return 0;
    // sequences are launched up to MAX_SEQS at a time, one launch after the other in the same room
    if (!pages_plan(B < alist::MAX_SEQS ? B : alist::MAX_SEQS, heads, T, max_pages, page_size, &p)) return -1;
    long long need = p.splits == 1 ? 0 : list_workspace((long long)p.nqb * heads * p.splits * 2, p.rows);
    if (B > alist::MAX_SEQS && B % alist::MAX_SEQS) {
        if (!pages_plan(B % alist::MAX_SEQS, heads, T, max_pages, page_size, &p)) return -1;
        const long long last = p.splits == 1 ? 0 : list_workspace((long long)p.nqb * heads * p.splits * 2, p.rows);
        need = last > need ? last : need;
    }
    return need;
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
    if (!map(&tq, q, ldq, g.q, g.qb) || !map(&tk, k, ldk, g.k, p.sub) || !map(&tv, v, ldv, g.k, p.sub))
        return cudaErrorInvalidValue;
    return launch_tiles<alist::BLOCKS>(tq, tk, tv, p, ws, ctx);
}

cudaError_t launch_attention_paged(const void* q, long long ldq, const KvPages& c, const int* lens, void* o,
                                   long long ldo, int B, int heads, int T, float* lse, void* ws, const LaunchCtx& ctx) {
    const uint64_t width = (uint64_t)heads * 128;
    for (int b0 = 0; b0 < B; b0 += alist::MAX_SEQS) {
        const int n = B - b0 < alist::MAX_SEQS ? B - b0 : alist::MAX_SEQS;
        ListParams p{};
        if (!pages_plan(n, heads, T, c.max_pages, c.page_size, &p)) return cudaErrorInvalidValue;
        p.table = c.table + b0 * c.table_ld;
        p.table_ld = c.table_ld;
        p.num_pages = c.num_pages;
        p.lens = lens + b0;
        p.o = reinterpret_cast<__nv_bfloat16*>(o) + (long long)b0 * T * ldo;
        p.ldo = ldo;
        p.lse = lse ? lse + (long long)b0 * heads * T : nullptr;
        const void* q0 = reinterpret_cast<const __nv_bfloat16*>(q) + (long long)b0 * T * ldq;
        cudaError_t e;
        if (T <= alist::ROWS_MOST) {
            e = T == 1 ? (p.row_warps == 4 ? launch_rows<1, 4>(q0, ldq, c, p, ws, ctx) : launch_rows<1, 8>(q0, ldq, c, p, ws, ctx))
                       : (p.row_warps == 4 ? launch_rows<2, 4>(q0, ldq, c, p, ws, ctx) : launch_rows<2, 8>(q0, ldq, c, p, ws, ctx));
        } else {
            const uint32_t group = 1u << p.log_group;
            CUtensorMap tq, tk, tv;
            if (!make_tmap_3d(&tq, q0, width, T, n, ldq, (uint64_t)ldq * T, 64, 128) ||
                !make_tmap_3d(&tk, c.k, width, c.page_size, c.num_pages, c.token_stride, c.page_stride, 64, group) ||
                !make_tmap_3d(&tv, c.v, width, c.page_size, c.num_pages, c.token_stride, c.page_stride, 64, group))
                return cudaErrorInvalidValue;
            e = launch_tiles<alist::PAGES>(tq, tk, tv, p, ws, ctx);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace wan
