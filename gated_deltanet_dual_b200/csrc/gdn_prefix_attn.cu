// gdn_prefix_attn.cu -- attention of a batch's newest tokens over a shared prefix and each
// sequence's own keys in a paged cache (gdn_prefix_attn of include/gdn_kvcache.h).
//
// softmax over a union of key sets is put together from the sets' parts: with
// m = max_s m_s,  out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s,  where a part holds, for its keys,
// the reference max m_s (log2 units), l_s = sum 2^(x - m_s) and o_s = sum 2^(x - m_s) v.  A row (n, l, h)
// has parts from the prefix (its keys cut into splits) and from its sequence's own keys (splits).
//
// The prefix is where the batch is read as one: for a key/value head, the N L (H / H_kv) query rows
// of ALL sequences are the rows of one matrix, so each prefix key is read once per 256 rows
// instead of once per sequence, and the product is a real matrix product for tcgen05.
//
// gdn_tile_attn_kernel -- one CTA = up to 256 query rows (two 128-row tiles) x a range of 128-key
// tiles of one key/value head.  Warp 8 loads K and V tiles page by page by TMA into a ring of
// five slots; warp 9 issues the MMAs; warps 0-3 and 4-7 are the softmax of row tile A and B (thread =
// row = TMEM lane).  The tensor pipe runs S = Q K^T and O += P V of one tile while the other tile's
// softmax runs: S_A, S_B, then per key tile PV_A, S_A(next), PV_B, S_B(next).  P (bf16) overwrites
// the first 64 TMEM columns of its S; MMAs of one issuing thread run in order, so S(next) follows
// the PV that reads it, and a thread that sees S(next) also knows that PV is done and may rescale O.
//
// gdn_warp_attn_kernel -- few query rows of a key list (L (H / H_kv) <= 16: a decode step): bound by
// reading K and V, and a 128-row tile would be padding.  One CTA = (key list, key/value head, split),
// with its own pages loaded by TMA into a ring of 64-key tiles.  Each of four warps takes 16 keys of
// every tile with a softmax state of its own, so warps never wait for one another inside the loop:
// S^T = K Q^T (mma m16n8k16, keys x rows, so 8 rows cost one column tile), P^T transposed in
// registers (movmatrix) into the B operand of O^T += V^T P^T.  The warps' states are joined at the end.
//
// gdn_attn_combine_kernel -- one warp per row joins the parts and rounds once to bf16.
//
// A sequence's last tile holds rows behind its last token, which may be anything: their scores are
// masked and their V rows are set to zero in shared memory (0 x NaN would be NaN in the MMA).  Among the
// L newest tokens of a causal call a value may be visible to some rows of the tile only:
// non-finite ones are set to zero too, and the combine kernel adds them to the rows that see them.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_internal.cuh"
#include "sm100.cuh"
#include "../../include/gdn_kvcache.h"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kTile = 128;                     // keys of a tile, rows of a row tile
constexpr int kRows = 2 * kTile;               // rows of a CTA
constexpr int kStages = 5;                     // K and V tiles in flight
constexpr int kTThreads = 320;
constexpr int kWKeys = 64;                     // gdn_warp_attn_kernel: keys of a tile (16 per warp)
constexpr int kWThreads = 160;                 // four warps of arithmetic and one that loads
constexpr int kWRows = 16;                     // most query rows
constexpr int kWStages = 3;
constexpr int kWMinTiles = 4;                  // a split of a sequence's own keys is not shorter
constexpr int kSms = 148;
constexpr int kMaxSplits = 64;
constexpr float kMargin = 8.f;                 // log2 units by which scores may pass the reference max
constexpr uint32_t kPWaitIters = 1u << 22;

struct PrefixParams {
    const __nv_bfloat16 *q, *v_cache;
    __nv_bfloat16 *out;
    const int32_t *prefix_pages, *block_table, *seq_lens;
    WorkspaceHeader *ws;
    int32_t *nonfinite;                        // [N]: the newest values of sequence n hold non-finite ones
    float2 *part_ml;                           // [parts][rows] (m, l)
    float *part_o;                             // [parts][rows][d]
    int64_t rows;                              // N L H
    int32_t N, L, H, Hkv, G, W, page, pages, prefix, causal;
    int32_t prefix_items, prefix_tiles, prefix_splits, own_tiles, own_splits;   // *_tiles: CTAs over the rows
    float scale_log2;
};

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}

// Own tokens of sequence n; -1 when the length is out of range.
__device__ __forceinline__ int own_len(const PrefixParams &P, int n) {
    const int s = P.seq_lens[n];
    return s < 0 || s > (int64_t)P.W * P.page ? -1 : s;
}

// What one CTA works on.
struct Item {
    int part, hk, row0, nrows, n;              // rows [row0, row0 + nrows) of the key/value head; n < 0: prefix
    int keys, t0, t1;                          // keys of the list, tiles [t0, t1) of it
    const int32_t *list;                       // page ids
};

// KEYS of a key tile, ROWS of a CTA; splits of own keys have at least MIN tiles.
template <int KEYS, int ROWS, int MIN>
__device__ __forceinline__ Item item_of(const PrefixParams &P, int b) {
    Item w;
    const int per_seq = P.L * P.G;
    if (b < P.prefix_items) {                  // row tiles fastest: those that run together share keys
        const int tile = b % P.prefix_tiles, rest = b / P.prefix_tiles;
        const int split = rest % P.prefix_splits;
        w.hk = rest / P.prefix_splits;
        w.part = split;
        w.n = -1;
        w.row0 = tile * ROWS;
        w.nrows = min(ROWS, P.N * per_seq - w.row0);
        w.keys = P.prefix;
        const int nt = (P.prefix + KEYS - 1) / KEYS;
        w.t0 = (int)((int64_t)nt * split / P.prefix_splits);
        w.t1 = (int)((int64_t)nt * (split + 1) / P.prefix_splits);
        w.list = P.prefix_pages;
    } else {
        b -= P.prefix_items;
        const int tile = b % P.own_tiles;
        b /= P.own_tiles;
        w.hk = b % P.Hkv;
        b /= P.Hkv;
        const int split = b % P.own_splits;
        w.n = b / P.own_splits;
        w.part = P.prefix_splits + split;
        w.row0 = w.n * per_seq + tile * ROWS;
        w.nrows = min(ROWS, per_seq - tile * ROWS);
        w.keys = max(own_len(P, w.n), 0);
        const int nt = (w.keys + KEYS - 1) / KEYS, per = max((nt + P.own_splits - 1) / P.own_splits, MIN);
        w.t0 = min(split * per, nt);
        w.t1 = min(w.t0 + per, nt);
        w.list = P.block_table + (int64_t)w.n * P.W;
    }
    return w;
}

// Global row (n, l, h) of row `row` of key/value head hk.
__device__ __forceinline__ int64_t row_of(const PrefixParams &P, int hk, int row) {
    const int nl = row / P.G;
    return (int64_t)nl * P.H + hk * P.G + (row - nl * P.G);
}

struct PrefixMaps {
    CUtensorMap k, v;                          // [P p, H_kv, d], box: 64 columns x 1 head x min(p, 64) rows
};

template <int D>
__global__ void __launch_bounds__(kTThreads, 1)
gdn_tile_attn_kernel(const __grid_constant__ PrefixParams P, const __grid_constant__ PrefixMaps M) {
    constexpr int kHalves = D / 64;
    constexpr int kTileBytes = kTile * D * 2;
    constexpr uint32_t T_S = 0, T_O = 256;     // TMEM columns: S of A, S of B, O of A, O of B (128 apart)
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    uint8_t *sm_q = sm, *sm_kv = sm + 2 * kTileBytes;
    __shared__ uint64_t full[kStages], empty[kStages], bar_q, bar_s[2], bar_p[2], bar_o[2], bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Item w = item_of<kTile, kRows, 1>(P, blockIdx.x);
    const int tiles = w.t1 - w.t0;
    float2 *ml = P.part_ml + w.part * P.rows;
    if (tiles == 0) {                          // an empty part: nothing visible
        for (int r = tid; r < w.nrows; r += kTThreads) ml[row_of(P, w.hk, w.row0 + r)] = make_float2(-INFINITY, 0.f);
        return;
    }
    const int two = w.nrows > kTile;           // row tile B is in use

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&bar_q, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_s[i], 1);
            mbar_init(&bar_p[i], 4);
            mbar_init(&bar_o[i], 1);
        }
        mbar_init(&bar_drain, 1);
        fence_mbar_init();
        s_abort = 0;
    }
    __syncwarp();
    if (warp == 0) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = s_tmem;

    // Bounded wait of a whole warp: false (in every lane) when it gave up, or another warp did.
    auto wait_ok = [&](uint64_t *bar, uint32_t parity, int where) {
        bool ok = false;
        for (uint32_t it = 0; it < kPWaitIters; ++it) {
            if ((ok = mbar_try_wait(bar, parity))) break;
            if ((it & 15) == 15 && *reinterpret_cast<volatile int *>(&s_abort)) break;
        }
        if (!ok && atomicExch(&s_abort, 1) == 0) {
            atomicExch(&P.ws->status, (int)GDN_ERR_TIMEOUT);
            atomicExch(&P.ws->timeout_where, where);
        }
        return __all_sync(0xffffffffu, ok) != 0;
    };

    if (warp == 8) {
        // ---------------------------------------------------------------- loads
        // lane = (half, box): a box is min(p, 64) rows of one page, 64 columns
        const int box_rows = min(P.page, 64), boxes = kTile / box_rows;
        const int box = lane % boxes, half = lane / boxes;
        const bool mine = half < kHalves;
        const int oob = P.pages * P.page;      // a row past the end: reads as zeros
        int issued = 0;
        for (; issued < 2 * tiles; ++issued) {
            const int j = w.t0 + (issued >> 1), slot = issued % kStages;
            const int key = j * kTile + box * box_rows;
            int row = oob;
            if (mine && key < w.keys) {
                const int id = w.list[key / P.page];
                if (id >= 0 && id < P.pages) row = id * P.page + key % P.page;
                else atomicCAS(&P.ws->status, 0, (int)GDN_ERR_INVALID_ARG);
            }
            if (issued >= kStages && !wait_ok(&empty[slot], (issued / kStages - 1) & 1, 1)) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], kTileBytes);
            __syncwarp();
            if (mine)
                tma_load_3d(sm_kv + slot * kTileBytes + half * (kTile * 128) + box * box_rows * 128,
                            (issued & 1) ? &M.v : &M.k, &full[slot], half * 64, w.hk, row);
            __syncwarp();
        }
        if (issued < 2 * tiles && lane == 0)   // gave up: the loads in flight still land
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait(&full[i % kStages], (i / kStages) & 1, kDrainWaitIters);
    } else if (warp == 9) {
        // ---------------------------------------------------------------- MMAs
        constexpr uint32_t idesc_s = make_idesc_bf16(128, 128, 0, 0);
        constexpr uint32_t idesc_o = make_idesc_bf16(128, D, 0, 1);
        const uint64_t dq = make_sdesc(smem_u32(sm_q), 16, 1024);
        auto score = [&](int t, int slot) {    // S_t = Q_t K^T
            const uint64_t dk = make_sdesc(smem_u32(sm_kv + slot * kTileBytes), 16, 1024);
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * (kTile * 128) + (kk & 3) * 32;
                mma_bf16(tb + T_S + 128 * t, dq + ((t * kTileBytes + off) >> 4), dk + (off >> 4), idesc_s, kk > 0);
            }
        };
        auto value = [&](int t, int slot, bool more) {   // O_t (+)= P_t V
            const uint64_t dv = make_sdesc(smem_u32(sm_kv + slot * kTileBytes), kTile * 128, 1024);
            for (int kk = 0; kk < 8; ++kk)
                mma_bf16_ts(tb + T_O + 128 * t, tb + T_S + 128 * t + kk * 8, dv + ((kk * 2048) >> 4), idesc_o, more || kk > 0);
        };
        bool ok = wait_ok(&bar_q, 0, 2) && wait_ok(&full[0], 0, 3);
        if (ok) {
            tc_fence_after();
            if (lane == 0) {
                score(0, 0);
                mma_commit(&bar_s[0]);
                if (two) {
                    score(1, 0);
                    mma_commit(&bar_s[1]);
                }
                mma_commit(&empty[0]);
            }
            __syncwarp();
        }
        for (int j = 0; ok && j < tiles; ++j) {
            const int iv = 2 * j + 1, ik = 2 * j + 2, sv = iv % kStages, sk = ik % kStages;
            const bool next = j + 1 < tiles;
            if (!(ok = wait_ok(&full[sv], (iv / kStages) & 1, 4))) break;
            // V rows that a row of the tile must not see
            const int key0 = (w.t0 + j) * kTile;
            uint8_t *v = sm_kv + sv * kTileBytes;
            const int last = min(kTile, w.keys - key0);          // rows [last, 128) are behind the list's end
            const int newest = (w.n >= 0 && P.causal) ? w.keys - (P.L - 1) : w.keys;
            if (last < kTile || newest < key0 + last) {
                for (int i = lane; i < (kTile - last) * (D / 8); i += 32) {
                    const int r = last + i / (D / 8), c = i % (D / 8);
                    *reinterpret_cast<uint4 *>(v + (c >> 3) * (kTile * 128) + sw128_off(r, c & 7)) = make_uint4(0, 0, 0, 0);
                }
                const int lo = max(newest - key0, 0);
                bool found = false;
                for (int i = lane; i < (last - lo) * (D / 8); i += 32) {
                    const int r = lo + i / (D / 8), c = i % (D / 8);
                    uint32_t *p = reinterpret_cast<uint32_t *>(v + (c >> 3) * (kTile * 128) + sw128_off(r, c & 7));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t x = p[e];
                        const bool a = (x & 0x7f80u) == 0x7f80u, b = (x & 0x7f800000u) == 0x7f800000u;
                        if (a) x &= 0xffff0000u;
                        if (b) x &= 0xffffu;
                        if (a || b) {
                            p[e] = x;
                            found = true;
                        }
                    }
                }
                if (found) P.nonfinite[w.n] = 1;
                fence_async_smem();
                __syncwarp();
            }
            if (next && !(ok = wait_ok(&full[sk], (ik / kStages) & 1, 5))) break;
            for (int t = 0; t <= two; ++t) {
                if (!(ok = wait_ok(&bar_p[t], j & 1, 6))) break;
                tc_fence_after();
                if (lane == 0) {
                    value(t, sv, j > 0);
                    if (t == two) mma_commit(&empty[sv]);
                    if (next) {
                        score(t, sk);
                        mma_commit(&bar_s[t]);
                        if (t == two) mma_commit(&empty[sk]);
                    } else {
                        mma_commit(&bar_o[t]);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) {                // gave up: the MMAs in flight still end
            mma_commit(&bar_drain);
            mbar_wait(&bar_drain, 0, kDrainWaitIters);
        }
    } else {
        // ---------------------------------------------------------------- queries, then softmax
        for (int i = tid; i < (two ? kRows : kTile) * (D / 8); i += 256) {
            const int r = i / (D / 8), c = i % (D / 8);
            uint4 u = make_uint4(0, 0, 0, 0);
            if (r < w.nrows) u = *reinterpret_cast<const uint4 *>(P.q + row_of(P, w.hk, w.row0 + r) * D + c * 8);
            *reinterpret_cast<uint4 *>(sm_q + (r >> 7) * kTileBytes + (c >> 3) * (kTile * 128) + sw128_off(r & 127, c & 7)) = u;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_q);

        const int t = warp >> 2, quad = warp & 3, r = tid;       // row of the CTA = thread
        const bool live = r < w.nrows;
        const bool warp_live = (warp << 5) < w.nrows;
        // keys [0, sees) are this row's
        int sees = live ? w.keys : 0;
        if (live && w.n >= 0 && P.causal) {
            const int l = ((w.row0 + r) / P.G) % P.L;
            sees = max(0, w.keys - (P.L - 1 - l));
        }
        const uint32_t ts = tmem_addr(tb, quad * 32, T_S + 128 * t), to = tmem_addr(tb, quad * 32, T_O + 128 * t);
        const float sl2 = P.scale_log2;
        float m_ref = -INFINITY, l_sum = 0.f;
        bool ok = true;
        if (t == 0 || two) {
            for (int j = 0; j < tiles; ++j) {
                if (!(ok = wait_ok(&bar_s[t], j & 1, 7))) break;
                __syncwarp();
                tc_fence_after();
                if (warp_live) {
                    float x[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, x[c]);
                    tmem_wait_ld();
                    const int hi = sees - (w.t0 + j) * kTile;    // columns [0, hi) are visible
                    float mt = -INFINITY;
                    if (hi >= kTile) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e) mt = fmaxf(mt, x[c][e]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                x[c][e] = 32 * c + e < hi ? x[c][e] : -INFINITY;
                                mt = fmaxf(mt, x[c][e]);
                            }
                    }
                    mt *= sl2;
                    float alpha = 1.f;
                    if (mt > m_ref + kMargin) {
                        alpha = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - mt);
                        m_ref = mt;
                    }
                    const float mu = m_ref == -INFINITY ? 0.f : m_ref;
                    if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            float o[32];
                            tmem_ld32(to + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= alpha;
                            tmem_st32(to + c0, o);
                        }
                    }
                    l_sum *= alpha;
                    float ls = 0.f;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float pk[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float p0 = ex2_approx(fmaf(x[2 * hf + e / 16][(2 * e) % 32], sl2, -mu));
                            const float p1 = ex2_approx(fmaf(x[2 * hf + e / 16][(2 * e) % 32 + 1], sl2, -mu));
                            ls += p0 + p1;
                            pk[e] = __uint_as_float(pack_bf2(p0, p1));
                        }
                        tmem_st32(ts + 32 * hf, pk);
                    }
                    l_sum += ls;
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_p[t]);
            }
            if (ok && (ok = wait_ok(&bar_o[t], 0, 8))) {
                __syncwarp();
                tc_fence_after();
                const int64_t row = live ? row_of(P, w.hk, w.row0 + r) : 0;
                if (m_ref == -INFINITY && l_sum != 0.f) m_ref = 0.f;   // every visible score is NaN: so is the row
                if (live) ml[row] = make_float2(m_ref, l_sum);
                float *po = P.part_o + (w.part * P.rows + row) * D;
                if (warp_live) {
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float o[32];
                        tmem_ld32(to + c0, o);
                        tmem_wait_ld();
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<float4 *>(po + c0 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tb, 512);
}

// ------------------------------------------------------------------------------------ few rows
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// c += a b: a 16 x 16 (row), b 16 x 8 (col), bf16 in, fp32 sums
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
constexpr int warp_smem() { return kWStages * 2 * kWKeys * D * 2 + 1024; }

// NT: column tiles of 8 rows.
template <int D, int NT>
__global__ void __launch_bounds__(kWThreads)
gdn_warp_attn_kernel(const __grid_constant__ PrefixParams P, const __grid_constant__ PrefixMaps M) {
    constexpr int kHalves = D / 64;
    constexpr int kHalfBytes = kWKeys * 128;
    constexpr int kTileBytes = kHalves * kHalfBytes;          // of K, and of V
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kWStages], empty[kWStages];
    __shared__ float2 s_ml[4][kWRows];
    __shared__ int s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Item w = item_of<kWKeys, kWRows, kWMinTiles>(P, blockIdx.x);
    const int tiles = w.t1 - w.t0;
    float2 *ml = P.part_ml + w.part * P.rows;
    if (tiles == 0) {                          // an empty part: nothing visible
        if (tid < w.nrows) ml[row_of(P, w.hk, w.row0 + tid)] = make_float2(-INFINITY, 0.f);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kWStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 4);
        }
        fence_mbar_init();
        s_abort = 0;
    }
    __syncthreads();

    auto wait_ok = [&](uint64_t *bar, uint32_t parity, int where) {
        bool ok = false;
        for (uint32_t it = 0; it < kPWaitIters; ++it) {
            if ((ok = mbar_try_wait(bar, parity))) break;
            if ((it & 15) == 15 && *reinterpret_cast<volatile int *>(&s_abort)) break;
        }
        if (!ok && atomicExch(&s_abort, 1) == 0) {
            atomicExch(&P.ws->status, (int)GDN_ERR_TIMEOUT);
            atomicExch(&P.ws->timeout_where, where);
        }
        return __all_sync(0xffffffffu, ok) != 0;
    };

    float acc[D / 16][NT][4];                  // O^T: (d, row)
    float m_ref[NT][2], l_sum[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][n][e] = 0.f;
        m_ref[n][0] = m_ref[n][1] = -INFINITY;
        l_sum[n][0] = l_sum[n][1] = 0.f;
    }

    if (warp == 4) {
        // lane = (value?, half, box): a box is min(p, 64) rows of one page, 64 columns
        const int box_rows = min(P.page, kWKeys), boxes = kWKeys / box_rows;
        const int box = lane % boxes, half = lane / boxes % kHalves, value = lane / (boxes * kHalves);
        const bool mine = value < 2;
        int issued = 0;
        for (; issued < tiles; ++issued) {
            const int slot = issued % kWStages;
            const int key = (w.t0 + issued) * kWKeys + box * box_rows;
            int row = P.pages * P.page;        // past the end: reads as zeros
            if (mine && key < w.keys) {
                const int id = w.list[key / P.page];
                if (id >= 0 && id < P.pages) row = id * P.page + key % P.page;
                else atomicCAS(&P.ws->status, 0, (int)GDN_ERR_INVALID_ARG);
            }
            if (issued >= kWStages && !wait_ok(&empty[slot], (issued / kWStages - 1) & 1, 11)) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2 * kTileBytes);
            __syncwarp();
            if (mine)
                tma_load_3d(sm + (2 * slot + value) * kTileBytes + half * kHalfBytes + box * box_rows * 128,
                            value ? &M.v : &M.k, &full[slot], half * 64, w.hk, row);
            __syncwarp();
        }
        if (issued < tiles && lane == 0)       // gave up: the loads in flight still land
            for (int i = max(0, issued - kWStages); i < issued; ++i)
                mbar_wait(&full[i % kWStages], (i / kWStages) & 1, kDrainWaitIters);
    } else {
        uint32_t qf[D / 16][NT][2];            // Q^T as B operands: row lane / 4, columns 2 (lane % 4) + {0, 1} (+ 8)
        int sees[NT][2];                       // keys [0, sees) are visible to rows 2 (lane % 4) + {0, 1}
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 8 + (lane >> 2);
            const uint32_t *src = reinterpret_cast<const uint32_t *>(P.q + row_of(P, w.hk, w.row0 + min(r, w.nrows - 1)) * D);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e) qf[kk][n][e] = r < w.nrows ? src[kk * 8 + e * 4 + (lane & 3)] : 0u;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = n * 8 + 2 * (lane & 3) + e;
                sees[n][e] = row < w.nrows ? w.keys : 0;
                if (row < w.nrows && w.n >= 0 && P.causal)
                    sees[n][e] = max(0, w.keys - (P.L - 1 - ((w.row0 + row) / P.G) % P.L));
            }
        }
        const float sl2 = P.scale_log2;
        // ldmatrix addresses inside this warp's 16 rows: K (row, 8 columns), V transposed
        const int krow = warp * 16 + (lane & 15), kchunk = lane >> 4;
        const int vrow = warp * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, vchunk = (lane >> 3) & 1;
        const uint32_t smb = smem_u32(sm);
        for (int i = 0; i < tiles; ++i) {
            const int slot = i % kWStages;
            if (!wait_ok(&full[slot], (i / kWStages) & 1, 12)) break;
            const int key0 = (w.t0 + i) * kWKeys + warp * 16;      // this warp's keys [key0, key0 + 16)
            if (key0 < w.keys) {
                const uint32_t kb = smb + 2 * slot * kTileBytes, vb = kb + kTileBytes;
                float s[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t a[4];
                    ldsm4(a, kb + (kk >> 2) * kHalfBytes + sw128_off(krow, (kk & 3) * 2 + kchunk));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816(s[n], a, qf[kk][n][0], qf[kk][n][1]);
                }
                // V rows that a row of the tile must not see (see the file comment)
                const int last = min(16, w.keys - key0);
                const int newest = (w.n >= 0 && P.causal) ? w.keys - (P.L - 1) : w.keys;
                if (last < 16 || newest < key0 + last) {
                    uint8_t *v = sm + (2 * slot + 1) * kTileBytes;
                    bool found = false;
                    for (int x = lane; x < 16 * (D / 8); x += 32) {
                        const int r = x / (D / 8), c = x % (D / 8);
                        uint32_t *p = reinterpret_cast<uint32_t *>(v + (c >> 3) * kHalfBytes + sw128_off(warp * 16 + r, c & 7));
                        if (r >= last) {
                            p[0] = p[1] = p[2] = p[3] = 0u;
                        } else if (key0 + r >= newest) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t y = p[e];
                                const bool a = (y & 0x7f80u) == 0x7f80u, b = (y & 0x7f800000u) == 0x7f800000u;
                                if (a) y &= 0xffff0000u;
                                if (b) y &= 0xffffu;
                                if (a || b) {
                                    p[e] = y;
                                    found = true;
                                }
                            }
                        }
                    }
                    if (found) P.nonfinite[w.n] = 1;
                    fence_async_smem();        // before the slot's next load
                    __syncwarp();
                }
                uint32_t pf[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + (lane >> 2) + (e >> 1) * 8;
                        s[n][e] = key < sees[n][e & 1] ? s[n][e] * sl2 : -INFINITY;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mt = fmaxf(s[n][e], s[n][e + 2]);
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                        const bool up = mt > m_ref[n][e] + kMargin;
                        if (__any_sync(0xffffffffu, up)) {
                            const float alpha = !up ? 1.f : m_ref[n][e] == -INFINITY ? 0.f : ex2_approx(m_ref[n][e] - mt);
                            if (up) m_ref[n][e] = mt;
                            l_sum[n][e] *= alpha;
#pragma unroll
                            for (int d0 = 0; d0 < D / 16; ++d0) {
                                acc[d0][n][e] *= alpha;
                                acc[d0][n][e + 2] *= alpha;
                            }
                        }
                        const float mu = m_ref[n][e] == -INFINITY ? 0.f : m_ref[n][e];
                        s[n][e] = ex2_approx(s[n][e] - mu);
                        s[n][e + 2] = ex2_approx(s[n][e + 2] - mu);
                        l_sum[n][e] += s[n][e] + s[n][e + 2];
                    }
                    pf[n][0] = transpose8x8(pack_bf2(s[n][0], s[n][1]));
                    pf[n][1] = transpose8x8(pack_bf2(s[n][2], s[n][3]));
                }
#pragma unroll
                for (int d0 = 0; d0 < D / 16; ++d0) {
                    uint32_t a[4];
                    ldsm4_trans(a, vb + (d0 >> 2) * kHalfBytes + sw128_off(vrow, (d0 & 3) * 2 + vchunk));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816(acc[d0][n], a, pf[n][0], pf[n][1]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
        }
        // this warp's (m, l): l summed over the keys of the eight lanes that share a row
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_sum[n][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (m_ref[n][e] == -INFINITY && l != 0.f) m_ref[n][e] = 0.f;   // every visible score is NaN: so is the row
                if (lane < 4) s_ml[warp][n * 8 + 2 * lane + e] = make_float2(m_ref[n][e], l);
            }
    }
    __syncthreads();                           // the ring is free: the warps' O^T go there, [warp][row][d]
    float *so = reinterpret_cast<float *>(sm);
    if (warp < 4) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = n * 8 + 2 * (lane & 3) + e;
                float m = -INFINITY;
#pragma unroll
                for (int x = 0; x < 4; ++x) m = fmaxf(m, s_ml[x][row].x);
                // a warp without a visible key has m = -inf and adds nothing (0 x anything is dropped)
                const bool none = m_ref[n][e] == -INFINITY;
                const float f = none ? 0.f : ex2_approx(m_ref[n][e] - m);
                float *dst = so + (warp * (NT * 8) + row) * D + (lane >> 2);
#pragma unroll
                for (int d0 = 0; d0 < D / 16; ++d0) {
                    dst[d0 * 16] = none ? 0.f : acc[d0][n][e] * f;
                    dst[d0 * 16 + 8] = none ? 0.f : acc[d0][n][e + 2] * f;
                }
            }
    }
    __syncthreads();
    if (tid < w.nrows) {
        float m = -INFINITY, l = 0.f;
        for (int x = 0; x < 4; ++x) m = fmaxf(m, s_ml[x][tid].x);
        for (int x = 0; x < 4; ++x)
            if (s_ml[x][tid].x != -INFINITY) l = fmaf(ex2_approx(s_ml[x][tid].x - m), s_ml[x][tid].y, l);
        ml[row_of(P, w.hk, w.row0 + tid)] = make_float2(m, l);
    }
    for (int x = tid; x < w.nrows * (D / 4); x += kWThreads) {
        const int row = x / (D / 4), c = x % (D / 4);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const float4 u = reinterpret_cast<const float4 *>(so)[(y * (NT * 8) + row) * (D / 4) + c];
            o.x += u.x, o.y += u.y, o.z += u.z, o.w += u.w;
        }
        reinterpret_cast<float4 *>(P.part_o + (w.part * P.rows + row_of(P, w.hk, w.row0 + row)) * D)[c] = o;
    }
}

// One warp per row (n, l, h): lane holds D / 32 columns.
template <int D>
__global__ void __launch_bounds__(256) gdn_attn_combine_kernel(const __grid_constant__ PrefixParams P, int parts) {
    constexpr int C = D / 32;
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (row >= P.rows) return;
    const int h = (int)(row % P.H), l = (int)(row / P.H % P.L), n = (int)(row / P.H / P.L);
    const int s = own_len(P, n);
    if (s < 0) {
        if (lane == 0) atomicCAS(&P.ws->status, 0, (int)GDN_ERR_INVALID_ARG);
        return;
    }
    float m = -INFINITY;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, P.part_ml[p * P.rows + row].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float acc[C], sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    if (m != -INFINITY) {
        for (int p = 0; p < parts; ++p) {
            const float2 a = P.part_ml[p * P.rows + row];
            if (a.x == -INFINITY) continue;
            const float f = ex2_approx(a.x - m);
            sum = fmaf(f, a.y, sum);
            const float *o = P.part_o + (p * P.rows + row) * D + lane * C;
            float x[C];
            if constexpr (C == 4) {
                const float4 u = *reinterpret_cast<const float4 *>(o);
                x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
            } else {
                const float2 u = *reinterpret_cast<const float2 *>(o);
                x[0] = u.x, x[1] = u.y;
            }
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = fmaf(f, x[c], acc[c]);
        }
        const float inv = 1.f / sum;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] *= inv;
        if (P.causal && P.L > 1 && P.nonfinite[n]) {   // set to zero in the product: they reach the rows that see them
            const int sees = max(0, s - (P.L - 1 - l));
            for (int key = max(0, s - (P.L - 1)); key < sees; ++key) {
                const int id = P.block_table[(int64_t)n * P.W + key / P.page];
                if (id < 0 || id >= P.pages) continue;
                const __nv_bfloat16 *v = P.v_cache + (((int64_t)id * P.page + key % P.page) * P.Hkv + h / P.G) * D + lane * C;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float x = __bfloat162float(v[c]);
                    if (!isfinite(x)) acc[c] += x;
                }
            }
        }
    }
    __nv_bfloat16 *out = P.out + row * D + lane * C;
    if constexpr (C == 4) *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf2(acc[0], acc[1]), pack_bf2(acc[2], acc[3]));
    else *reinterpret_cast<uint32_t *>(out) = pack_bf2(acc[0], acc[1]);
}

// ------------------------------------------------------------------------------------ host
PFN_cuTensorMapEncodeTiled_v12000 prefix_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool cache_map(CUtensorMap *m, const void *ptr, const gdn_prefix_attn_desc *D) {
    auto enc = prefix_encoder();
    if (!enc) return false;
    const cuuint64_t d = D->head_dim, hk = D->num_kv_heads;
    cuuint64_t dims[3] = {d, hk, (cuuint64_t)D->num_pages * D->page_size};
    cuuint64_t strides[2] = {d * 2, hk * d * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)std::min(D->page_size, 64)};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool desc_ok(const gdn_prefix_attn_desc *D) {
    return D && D->num_seqs >= 1 && D->num_tokens >= 1 && D->num_heads >= 1 && D->num_kv_heads >= 1 && D->head_dim >= 1 &&
           D->page_size >= 1 && D->num_pages >= 1 && D->table_width >= 0 && D->prefix_len >= 0 &&
           (D->causal == 0 || D->causal == 1) && (D->dtype == GDN_BF16 || D->dtype == GDN_FP32) &&
           (D->scale == 0.f || (D->scale > 0.f && std::isfinite(D->scale))) && D->num_heads % D->num_kv_heads == 0 &&
           (int64_t)D->num_pages * D->page_size <= INT32_MAX && (int64_t)D->table_width * D->page_size <= INT32_MAX - kTile &&
           D->prefix_len <= INT32_MAX - kTile;
}

bool desc_supported(const gdn_prefix_attn_desc *D) {
    const int p = D->page_size;
    return D->dtype == GDN_BF16 && (D->head_dim == 64 || D->head_dim == 128) &&
           (p == 16 || p == 32 || p == 64 || p == 128 || p == 256) &&
           (int64_t)D->num_seqs * D->num_tokens * D->num_heads <= INT32_MAX / 2;
}

// How a call is cut into CTAs and parts.
struct Plan {
    int64_t rows;
    bool prefix_warp, own_warp;                // by gdn_warp_attn_kernel (else gdn_tile_attn_kernel)
    int prefix_tiles, prefix_splits, own_tiles, own_splits, parts;
    int64_t prefix_items, own_items;
    size_t off_nonfinite, off_ml, off_o, bytes;
};

// Splits of `tiles` key tiles over `base` equal work items: waves of CTAs times a CTA's tiles, three more
// for its set-up and its part of the combine step.
int best_split(int64_t base, int64_t tiles) {
    int best = 1;
    double cost = 1e300;
    for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
        const double waves = (double)((base * s + kSms - 1) / kSms);
        const double c = waves * ((double)((tiles + s - 1) / s) + 3.0);
        if (c < cost * 0.999) cost = c, best = s;
    }
    return best;
}

// The same for gdn_warp_attn_kernel, whose CTAs share an SM and whose lists differ in length: four
// CTAs for each place on the GPU while no split gets shorter than its least.
int warp_split(int64_t base, int64_t keys) {
    const int64_t most = (keys + kWKeys * kWMinTiles - 1) / (kWKeys * kWMinTiles);
    return (int)std::max<int64_t>(1, std::min<int64_t>({(4 * 2 * kSms + base - 1) / base, most, kMaxSplits}));
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

Plan plan_of(const gdn_prefix_attn_desc *D) {
    Plan p;
    const int64_t G = D->num_heads / D->num_kv_heads, per_seq = D->num_tokens * G;
    p.rows = (int64_t)D->num_seqs * D->num_tokens * D->num_heads;
    p.prefix_warp = D->num_seqs * per_seq <= kWRows;
    p.own_warp = per_seq <= kWRows;
    const int64_t own_room = (int64_t)D->table_width * D->page_size;
    p.prefix_tiles = p.prefix_warp ? 1 : (int)((D->num_seqs * per_seq + kRows - 1) / kRows);
    p.own_tiles = p.own_warp ? 1 : (int)((per_seq + kRows - 1) / kRows);
    const int64_t prefix_base = (int64_t)D->num_kv_heads * p.prefix_tiles;
    const int64_t own_base = (int64_t)D->num_seqs * D->num_kv_heads * p.own_tiles;
    p.prefix_splits = !D->prefix_len ? 0 : p.prefix_warp ? warp_split(prefix_base, D->prefix_len)
                                                         : best_split(prefix_base, ((int64_t)D->prefix_len + kTile - 1) / kTile);
    p.own_splits = !own_room ? 0 : p.own_warp ? warp_split(own_base, own_room) : best_split(own_base, (own_room + kTile - 1) / kTile);
    p.prefix_items = (int64_t)D->num_kv_heads * p.prefix_tiles * p.prefix_splits;
    p.own_items = (int64_t)D->num_seqs * D->num_kv_heads * p.own_tiles * p.own_splits;
    p.parts = p.prefix_splits + p.own_splits;
    p.off_nonfinite = sizeof(WorkspaceHeader);
    p.off_ml = p.off_nonfinite + round256((size_t)D->num_seqs * 4);
    p.off_o = p.off_ml + round256((size_t)p.parts * p.rows * 8);
    p.bytes = p.off_o + round256((size_t)p.parts * p.rows * D->head_dim * 4);
    return p;
}

template <int D>
constexpr int tile_smem() { return (2 + kStages) * kTile * D * 2 + 1024; }

// Raises the kernels' dynamic shared memory limits, once per device.
template <int D>
cudaError_t prepare_device() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    e = cudaFuncSetAttribute(gdn_tile_attn_kernel<D>, attr, tile_smem<D>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_warp_attn_kernel<D, 1>, attr, warp_smem<D>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_warp_attn_kernel<D, 2>, attr, warp_smem<D>());
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// One launch over the prefix's items, the own keys' items, or both.
template <int D>
cudaError_t launch_parts(PrefixParams P, const PrefixMaps &maps, const Plan &plan, bool warp, bool prefix, bool own,
                         cudaStream_t st) {
    P.prefix_items = prefix ? (int32_t)plan.prefix_items : 0;
    const int64_t items = P.prefix_items + (own ? plan.own_items : 0);
    if (items == 0) return cudaSuccess;
    if (!warp) {
        gdn_tile_attn_kernel<D><<<(unsigned)items, kTThreads, tile_smem<D>(), st>>>(P, maps);
    } else if ((prefix ? (int64_t)P.N : 1) * P.L * P.G <= 8) {
        gdn_warp_attn_kernel<D, 1><<<(unsigned)items, kWThreads, warp_smem<D>(), st>>>(P, maps);
    } else {
        gdn_warp_attn_kernel<D, 2><<<(unsigned)items, kWThreads, warp_smem<D>(), st>>>(P, maps);
    }
    return cudaGetLastError();
}

template <int D>
gdn_status launch(const PrefixParams &P, const PrefixMaps &maps, const Plan &plan, cudaStream_t st) {
    if (prepare_device<D>() != cudaSuccess) return GDN_ERR_CUDA;
    if (plan.prefix_warp == plan.own_warp) {
        if (launch_parts<D>(P, maps, plan, plan.own_warp, true, true, st) != cudaSuccess) return GDN_ERR_CUDA;
    } else if (launch_parts<D>(P, maps, plan, plan.prefix_warp, true, false, st) != cudaSuccess ||
               launch_parts<D>(P, maps, plan, plan.own_warp, false, true, st) != cudaSuccess) {
        return GDN_ERR_CUDA;
    }
    gdn_attn_combine_kernel<D><<<(unsigned)((plan.rows + 7) / 8), 256, 0, st>>>(P, plan.parts);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_prefix_attn_workspace_size(const gdn_prefix_attn_desc *desc) {
    if (!desc_ok(desc) || !desc_supported(desc)) return 0;
    return plan_of(desc).bytes;
}

extern "C" gdn_status gdn_prefix_attn(const gdn_prefix_attn_desc *D, const void *q, const void *k_cache,
                                      const void *v_cache, const int32_t *prefix_pages, const int32_t *block_table,
                                      const int32_t *seq_lens, void *out, void *workspace, size_t workspace_bytes,
                                      gdn_stream_t stream) {
    if (!desc_ok(D)) return GDN_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !seq_lens || !out || !workspace || (D->prefix_len > 0 && !prefix_pages) ||
        (D->table_width > 0 && !block_table))
        return GDN_ERR_INVALID_ARG;
    auto off = [](const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
    if (off(q, 16) || off(k_cache, 16) || off(v_cache, 16) || off(out, 16) || off(prefix_pages, 4) || off(block_table, 4) ||
        off(seq_lens, 4) || off(workspace, 256))
        return GDN_ERR_ALIGNMENT;
    if (!desc_supported(D)) return GDN_ERR_UNSUPPORTED;
    const Plan plan = plan_of(D);
    if (plan.prefix_items + plan.own_items > INT32_MAX) return GDN_ERR_UNSUPPORTED;
    if (workspace_bytes < plan.bytes) return GDN_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    PrefixParams P = {};
    P.q = static_cast<const __nv_bfloat16 *>(q);
    P.v_cache = static_cast<const __nv_bfloat16 *>(v_cache);
    P.out = static_cast<__nv_bfloat16 *>(out);
    P.prefix_pages = prefix_pages, P.block_table = block_table, P.seq_lens = seq_lens;
    P.ws = reinterpret_cast<WorkspaceHeader *>(ws);
    P.nonfinite = reinterpret_cast<int32_t *>(ws + plan.off_nonfinite);
    P.part_ml = reinterpret_cast<float2 *>(ws + plan.off_ml);
    P.part_o = reinterpret_cast<float *>(ws + plan.off_o);
    P.rows = plan.rows;
    P.N = D->num_seqs, P.L = D->num_tokens, P.H = D->num_heads, P.Hkv = D->num_kv_heads, P.G = P.H / P.Hkv;
    P.W = D->table_width, P.page = D->page_size, P.pages = D->num_pages, P.prefix = D->prefix_len, P.causal = D->causal;
    P.prefix_tiles = plan.prefix_tiles, P.prefix_splits = plan.prefix_splits;
    P.own_tiles = plan.own_tiles, P.own_splits = plan.own_splits;
    const double scale = D->scale > 0.f ? D->scale : 1.0 / std::sqrt((double)D->head_dim);
    P.scale_log2 = (float)(1.4426950408889634 * scale);
    PrefixMaps maps;
    if (!cache_map(&maps.k, k_cache, D) || !cache_map(&maps.v, v_cache, D)) return GDN_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(ws, 0, plan.off_ml, st) != cudaSuccess) return GDN_ERR_CUDA;
    return D->head_dim == 64 ? launch<64>(P, maps, plan, st) : launch<128>(P, maps, plan, st);
}
