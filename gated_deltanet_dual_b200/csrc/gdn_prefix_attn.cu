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
// gdn_tile_attn_kernel -- one CTA = up to 256 query rows (row tiles A and B of 128) x a range of 128-key
// tiles of one key/value head.  Warp 16 loads K and V tiles page by page by TMA into a ring, warp 17 issues
// S = Q K^T, warp 19 cleans V rows that must not be seen and issues O += P V; warps 0-7 and 8-15 are the softmax of
// A and B.  A row (TMEM lane) has two threads, each with 64 of a tile's 128 scores: they share the maximum only
// when it moves.  S_A and S_B take turns in the same TMEM columns, which are free as soon as the scores are in
// registers; P (bf16) has columns of its own per row tile, so S(next) runs while this tile's exponentials
// do.  In its loop bound by the tensor pipe: a tile step of 256 rows takes 1.6 us, of which the products take 1.45 at the
// pipe's measured rate.  256 requests of 4 query heads per key/value head over 16384 prefix keys take 74 us: 44 of tile
// steps on all SMs (the products 40), the rest a CTA's start and end (12 us) and the uneven last wave.
//
// gdn_warp_attn_kernel -- few query rows of a key list (L (H / H_kv) <= 16: a decode step): bound by
// reading K and V, and a 128-row tile would be padding.  One CTA = (key list, key/value head, split),
// with its own pages loaded by TMA into a ring of 64-key tiles.  Each of four warps takes 16 keys of
// every tile with a softmax state of its own, so warps never wait for one another inside the loop:
// S^T = K Q^T (mma m16n8k16, keys x rows, so 8 rows cost one column tile), P^T transposed in
// registers (movmatrix) into the B operand of O^T += V^T P^T.  The warps' states are joined at the end.  32
// requests of up to 16384 own tokens, 32 query heads on 8: 184 us, the time of one read at 6.46 TB/s; of short
// lists the start and end show: 64 requests of up to 1024 tokens 33 us, where one read takes 21.
//
// P is rounded to bf16 for the second product: each term of a row's sum is off by at most 2^-8 of itself, in the
// size of the output's own rounding; its sum l is taken before the rounding, in fp32, as is everything else.
//
// gdn_attn_combine_kernel -- one warp per row joins the parts and rounds once to bf16.  Bound by latency (the wait
// for the parts, then two dependent reads from L2): about 4 us of a call.
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
constexpr int kTThreads = 640;                 // 16 softmax warps, load, S, idle, P V (register shares go by four warps)
// Registers a thread: the launch gives 96 (65536 / 640, in eights); the softmax warps hold half a row of
// S and take what the load and MMA warps give up.  The compiler spills 32 bytes a thread at d = 128 (24 at 64; 14 and
// 12 stores of 4 bytes, 36 and 26 loads, in all roles together).
constexpr int kRegsLaunch = 96, kRegsSoftmax = 104, kRegsOther = 56;
static_assert(4 * kRegsSoftmax + kRegsOther <= 5 * kRegsLaunch, "a warpgroup would wait for registers for ever");
constexpr int kWKeys = 64;                     // gdn_warp_attn_kernel: keys of a tile (16 per warp)
constexpr int kWThreads = 160;                 // four warps of arithmetic and one that loads
constexpr int kWRows = 16;                     // most query rows
constexpr int kWMinTiles = 4;                  // a split of a sequence's own keys is not shorter
constexpr int kSms = 148;
constexpr int kMaxSplits = 64;
constexpr float kMargin = 8.f;                 // log2 units by which scores may pass the reference max
constexpr uint32_t kPWaitIters = 1u << 22;

// An item's status word: a gdn_status, a mark, and from bit 16 on the site of a wait that gave up.
constexpr int kItemNonfinite = 1 << 8;         // among the sequence's newest values were non-finite ones

struct PrefixParams {
    const __nv_bfloat16 *q, *v_cache;
    __nv_bfloat16 *out;
    const int32_t *prefix_pages, *block_table, *seq_lens;
    WorkspaceHeader *ws;
    int32_t *item_status;                      // [items]: what went wrong in a CTA, see kItemNonfinite
    float2 *part_ml;                           // [parts][rows] (m, l)
    float *part_o;                             // [parts][rows][d]
    int64_t rows;                              // N L H
    int32_t N, L, H, Hkv, G, W, page, pages, prefix, causal;
    int32_t first_item, items_of_prefix;       // this launch's first item; items [0, items_of_prefix) are the prefix's
    int32_t prefix_tiles, prefix_splits, own_tiles, own_splits;   // *_tiles: CTAs over the rows
    int32_t prefix_rows, own_rows;             // rows of such a CTA
    float scale_log2;
    uint32_t wait_iters;                       // polls of a wait in the test instantiations
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

// 32 lanes x 16 consecutive 32-bit TMEM columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
          "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// 16 bytes global -> shared, asynchronously; zeros where !in (nothing is read).
__device__ __forceinline__ void cp_async16_or_zero(void *dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Bounded wait in one piece: true once the phase with this parity is complete.
__device__ __forceinline__ bool mbar_wait_some(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 0;\n\t"
        "again:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra done;\n\t"
        "add.u32 n, n, 1;\n\t"
        "setp.lt.u32 q, n, 16;\n\t"
        "@q bra again;\n\t"
        "done:\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Two fp32 values in one 64-bit register, and the packed arithmetic on them.
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_of(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_get(f2 x, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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

// Dependent launches.  A call's kernels overlap: each lets the next one's CTAs start as soon as its own have
// all started.  The first kernel of a call waits for the work before it (the inputs, an earlier call's use of the
// workspace) and only then lets the next one start, so the second kernel may read inputs and write its parts at
// once.  The combine kernel waits for the second kernel, whose last CTA waits for the first one before it ends (if
// every CTA did, the first ones to be done would keep their SMs from those that have not started).
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_end() {
    if (blockIdx.x == gridDim.x - 1) grid_wait();
}

// KEYS of a key tile, ROWS of a CTA; splits of own keys have at least MIN tiles.
template <int KEYS, int ROWS, int MIN>
__device__ __forceinline__ Item item_of(const PrefixParams &P, int b) {
    Item w;
    const int per_seq = P.L * P.G;
    if (b < P.items_of_prefix) {                  // row tiles fastest: those that run together share keys
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
        b -= P.items_of_prefix;
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

// Half a row of S, x (-inf where a key is not visible), to P = 2^(x scale - m_ref) as bf16 pairs in the TMEM
// columns [tp, tp + 32), which may be written once free() has returned: ls = the sum of P, mt = the largest
// x in log2 units.  Bound by the exponential unit (8 clocks a warp instruction); taking a share of the
// exponentials as polynomials on the FMA pipe gained nothing.
template <typename FREE>
__device__ __forceinline__ void softmax_half(const float (&x)[2][32], float scale, float m_ref, uint32_t tp, float &ls,
                                             float &mt, const FREE &free) {
    const float mu = m_ref == -INFINITY ? 0.f : m_ref;
    const f2 scale2 = f2_of(scale, scale), shift2 = f2_of(-mu, -mu);
    f2 sum[4] = {0, 0, 0, 0};
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float x0 = x[c][2 * e], x1 = x[c][2 * e + 1];
            mx[e & 3] = fmaxf(mx[e & 3], fmaxf(x0, x1));
            float p0, p1;
            f2_get(f2_fma(f2_of(x0, x1), scale2, shift2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            sum[e & 3] = f2_add(sum[e & 3], f2_of(p0, p1));
            pk[e] = pack_bf2(p0, p1);
        }
        if (c == 0) free();
        tmem_st16(tp + 16 * c, pk);
    }
    float ls1;
    f2_get(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), ls, ls1);
    ls += ls1;
    mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
}

struct PrefixMaps {
    CUtensorMap k, v;                          // [P p, H_kv, d], box: 64 columns x 1 head x min(p, 64) rows
};

// TW: the test instantiation, whose waits poll with the caller's bound (gdn_prefix_attn_test_wait_limit).
template <int D, bool TW>
__global__ void __launch_bounds__(kTThreads, 1)
gdn_tile_attn_kernel(const __grid_constant__ PrefixParams P, const __grid_constant__ PrefixMaps M) {
    constexpr int kHalves = D / 64;
    constexpr int kTileBytes = kTile * D * 2;
    constexpr uint32_t T_S = 0, T_P = 128, T_O = 256;    // TMEM columns: S; P of A and B (64 apart); O of A and B (128 apart)
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    uint8_t *sm_q = sm, *sm_kv = sm + 2 * kTileBytes;
    __shared__ uint64_t full[kStages], empty[kStages];
    // S of A / B is complete; it is in registers; P of A / B is written; P V is done
    __shared__ uint64_t bar_s[2], bar_r[2], bar_p[2], bar_o[2], bar_drain[2];
    __shared__ float s_pair[kRows];            // between a row's two threads: maxima, at the end a sum
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_status;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int item = P.first_item + blockIdx.x;
    if (P.first_item == 0) grid_wait();
    grid_next();
    if (item == 0 && tid == 0) P.ws->status = P.ws->timeout_where = 0;
    const Item w = item_of<kTile, kRows, 1>(P, item);
    const int tiles = w.t1 - w.t0;
    float2 *ml = P.part_ml + w.part * P.rows;
    if (tiles == 0) {                          // an empty part: nothing visible
        for (int r = tid; r < w.nrows; r += kTThreads) ml[row_of(P, w.hk, w.row0 + r)] = make_float2(-INFINITY, 0.f);
        if (tid == 0) P.item_status[item] = 0;
        grid_end();
        return;
    }
    const int two = w.nrows > kTile;           // row tile B is in use

    // The ring's order is the order of use, K0 K1 V0 K2 V1 ... V(last): K(j) has place 2 j - 1 (K0: 0), V(j) 2 j + 2, the
    // last V 2 tiles - 1.  Warp 17 waits for the K tiles and warp 19 for the V tiles, each by parity, which is right only
    // if the slot's use before, kStages places back, has landed.  It has:
    //   at K(j), warp 17 has seen S(j - 2) taken into registers, which the softmax warps do once P V(j - 4) is done: K(j - 1)
    //   and V(j - 4) have landed, places 2 j - 3 and 2 j - 6, and what lies before each of the same kind;
    //   at V(j), warp 19 has seen P(j - 1) written: V(j - 1) and K(j - 1), places 2 j and 2 j - 3, and so on.
    // Four places or more back all is covered, at three it would not be.
    static_assert(kStages >= 4, "a wait for a slot's use could pass on the parity of the use before the last");
    // Loads tile i of the ring (warp 16): lane = (half, box), a box is min(p, 64) rows of one page, 64 columns; rows past
    // the end read as zeros.
    const int box_rows = min(P.page, 64), boxes = kTile / box_rows, box = lane % boxes, half_of = lane / boxes;
    // This lane's cache row in key tile j, for K and again for V; the page ids of the tile after are on their way.
    int id_next = 0, rows_of[2] = {0, 0};
    bool id_wanted = false;                    // any id may stand in the table: whether there is one is kept apart
    auto fetch_id = [&](int j) {
        const int key = (w.t0 + j) * kTile + box * box_rows;
        id_wanted = half_of < kHalves && j < tiles && key < w.keys;
        if (id_wanted) id_next = w.list[key / P.page];
    };
    auto load = [&](int i) {
        const bool value = i > 0 && ((i & 1) == 0 || i == 2 * tiles - 1);
        const int j = value ? (i == 2 * tiles - 1 ? tiles - 1 : i / 2 - 1) : (i + 1) / 2;
        const int slot = i % kStages;
        if (!value) {
            const int id = id_next;
            int row = P.pages * P.page;        // past the end: reads as zeros
            if (id_wanted) {
                if (id >= 0 && id < P.pages) row = id * P.page + ((w.t0 + j) * kTile + box * box_rows) % P.page;
                else atomicOr(&s_status, (int)GDN_ERR_INVALID_ARG);
            }
            if (j & 1) rows_of[1] = row;
            else rows_of[0] = row;
            fetch_id(j + 1);
        }
        const int row = j & 1 ? rows_of[1] : rows_of[0];
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], kTileBytes);
        __syncwarp();
        if (half_of < kHalves)
            tma_load_3d(sm_kv + slot * kTileBytes + half_of * (kTile * 128) + box * box_rows * 128, value ? &M.v : &M.k,
                        &full[slot], half_of * 64, w.hk, row);
        __syncwarp();
    };
    if (warp == 16) {
        fetch_id(0);
        if (lane == 0) {
            for (int i = 0; i < kStages; ++i) {
                mbar_init(&full[i], 1);
                mbar_init(&empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bar_s[i], 1);
                mbar_init(&bar_r[i], 8);
                mbar_init(&bar_p[i], 8);
                mbar_init(&bar_o[i], 1);
                mbar_init(&bar_drain[i], 1);
            }
            fence_mbar_init();
            fence_async_smem();
            s_abort = s_status = 0;
        }
        __syncwarp();
        for (int i = 0; i < min(kStages, 2 * tiles); ++i) load(i);         // beside the queries' loads
    } else if (warp == 17) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    } else if (warp < 16) {
        // queries: D / 8 chunks of 16 bytes a row, a pass covers 512 / (D / 8) rows; asynchronous copies in a short
        // loop (a launch starts with cold instruction caches); rows past the last are zeros
        constexpr int kChunks = D / 8, kPass = 512 / kChunks;
        const int c = tid % kChunks;
        int r = tid / kChunks;
        int nl = (w.row0 + r) / P.G, g = (w.row0 + r) - nl * P.G;         // (n, l) and head of the row
        const int dn = kPass / P.G, dg = kPass - dn * P.G;               // the same of kPass rows
        const __nv_bfloat16 *head = P.q + (int64_t)w.hk * P.G * D + c * 8;
        uint8_t *dst = sm_q + (c >> 3) * (kTile * 128) + sw128_off(r, c & 7);
#pragma unroll 1
        for (int i = 0; i < (1 + two) * kTile / kPass; ++i) {
            const bool in = r < w.nrows;
            cp_async16_or_zero(dst + (r >> 7) * (kTileBytes - kTile * 128), head + (in ? ((int64_t)nl * P.H + g) * D : 0), in);
            r += kPass, dst += kPass * 128, nl += dn;
            if ((g += dg) >= P.G) g -= P.G, ++nl;
        }
        cp_async_commit();
        cp_async_wait_all();
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = s_tmem;

    // Bounded wait.  A wait that gives up marks the CTA as stopping and returns; every further wait gives up at
    // once.  Loads and products stop at the end of the key tile; the softmax warps, which meet at the barriers of
    // their pairs, run through their tiles (on unspecified data) and write nothing.
    auto stopped = [&] { return *reinterpret_cast<volatile int *>(&s_abort) != 0; };
    auto wait = [&](uint64_t *bar, uint32_t parity, int where) {
        if constexpr (TW) {
            if (stopped() || mbar_poll(bar, parity, P.wait_iters)) return;
        } else {
            if (mbar_try_wait(bar, parity)) return;
            for (uint32_t it = 0; it < kPWaitIters / 16; ++it) {
                if (mbar_wait_some(bar, parity)) return;
                if (stopped()) return;
            }
        }
        if (atomicExch(&s_abort, 1) == 0) atomicExch(&s_status, (int)GDN_ERR_TIMEOUT | where << 16);
    };
    // V rows from key `newest` on are not for every query row (see the file comment): warp 19 cleans their tiles
    const int newest = (w.n >= 0 && P.causal) ? w.keys - (P.L - 1) : w.keys;

    // one instruction for all four warps of a warpgroup: those of the last take different roles behind it
    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 16) {
            // ---------------------------------------------------------------- loads
            int issued = min(kStages, 2 * tiles);
            for (; issued < 2 * tiles; ++issued) {
                wait(&empty[issued % kStages], (issued / kStages - 1) & 1, 1);
                __syncwarp();
                if (__any_sync(0xffffffffu, stopped())) break;     // the slot may still be in use
                load(issued);
            }
            if (__any_sync(0xffffffffu, stopped()) && lane == 0)   // gave up: the loads in flight still land
                for (int i = max(0, issued - kStages); i < issued; ++i)
                    mbar_wait(&full[i % kStages], (i / kStages) & 1, kDrainWaitIters);
        } else if (warp == 17 || warp == 19) {
            // ---------------------------------------------------------------- products: S (warp 17), P V (warp 19)
            // Two streams, so that one's products run while the other waits on a barrier; warp-uniform, with few
            // instructions between the products (a single thread's chain of address arithmetic and branches
            // cost more than the products that it fed).
            constexpr uint32_t kStep = kTileBytes >> 4;
            int slot = 0, left = tiles;
            uint32_t phase = 0;
            auto advance = [&](int n) {            // n tiles on in the ring
                slot += n;
                if (slot >= kStages) slot -= kStages, phase ^= 1;
            };
            if (warp == 17) {
                constexpr uint32_t idesc = make_idesc_bf16(128, 128, 0, 0);
                const uint64_t dq = make_sdesc(smem_u32(sm_q), 16, 1024), dk = make_sdesc(smem_u32(sm_kv), 16, 1024);
                uint32_t odd = 0;                  // parity of the key tile
                for (int j = 0; j < tiles; ++j, odd ^= 1) {
                    wait(&full[slot], phase, 2);
                    for (int t = 0; t <= two; ++t) {
                        // the S before this one (of the other row tile, or of this one) is in registers
                        if (t == 1) wait(&bar_r[0], odd, 3);
                        else if (j > 0) wait(&bar_r[two], odd ^ 1, 3);
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = ((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
                                mma_bf16(tb + T_S, dq + t * kStep + off, dk + slot * kStep + off, idesc, kk > 0);
                            }
                            mma_commit(&bar_s[t]);
                            if (t == two) mma_commit(&empty[slot]);
                        }
                        __syncwarp();
                    }
                    advance(j == 0 ? 1 : 2);
                    if (__any_sync(0xffffffffu, stopped())) break;
                }
            } else {
                constexpr uint32_t idesc = make_idesc_bf16(128, D, 0, 1);
                const uint64_t dv = make_sdesc(smem_u32(sm_kv), kTile * 128, 1024);
                int end = (w.t0 + 1) * kTile;
                slot = tiles > 1 ? 2 : 1;
                for (int j = 0; j < tiles; ++j, end += kTile) {
                    wait(&full[slot], phase, 4);
                    if (end > newest) {
                        const int key0 = end - kTile;
                        uint8_t *v = sm_kv + slot * kTileBytes;
                        const int last = min(kTile, w.keys - key0);          // rows [last, 128) are behind the list's end
                        for (int i = lane; i < (kTile - last) * (D / 8); i += 32) {
                            const int r = last + i / (D / 8), c = i % (D / 8);
                            *reinterpret_cast<uint4 *>(v + (c >> 3) * (kTile * 128) + sw128_off(r, c & 7)) = make_uint4(0, 0, 0, 0);
                        }
                        const int lo = max(newest - key0, 0);                // rows [lo, last) are visible to some rows only
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
                        if (found) atomicOr(&s_status, kItemNonfinite);
                        fence_async_smem();
                        __syncwarp();
                    }
                    for (int t = 0; t <= two; ++t) {
                        wait(&bar_p[t], j & 1, 6);
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_bf16_ts(tb + T_O + 128 * t, tb + T_P + 64 * t + kk * 8, dv + slot * kStep + kk * 128, idesc,
                                            j > 0 || kk > 0);
                            mma_commit(&bar_o[t]);
                            if (t == two) mma_commit(&empty[slot]);
                        }
                        __syncwarp();
                    }
                    advance(--left > 1 ? 2 : 1);   // the last V follows the one before it
                    if (__any_sync(0xffffffffu, stopped())) break;
                }
            }
            if (__any_sync(0xffffffffu, stopped()) && elect_one()) {       // gave up: the MMAs in flight still end
                mma_commit(&bar_drain[warp == 19]);
                mbar_wait(&bar_drain[warp == 19], 0, kDrainWaitIters);
            }
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int t = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
        const int r = t * kTile + quad * 32 + lane;                            // row of the CTA
        const int pair = 1 + t * 4 + quad;                                     // named barrier of the rows' two warps
        const bool live = r < w.nrows;
        const bool warp_live = t * kTile + quad * 32 < w.nrows;
        // keys [0, sees) are this row's
        int sees = live ? w.keys : 0;
        if (live && w.n >= 0 && P.causal) {
            const int l = ((w.row0 + r) / P.G) % P.L;
            sees = max(0, w.keys - (P.L - 1 - l));
        }
        const uint32_t ts = tmem_addr(tb, quad * 32, T_S + 64 * half);                     // this thread's half of S,
        const uint32_t tp = tmem_addr(tb, quad * 32, T_P + 64 * t + 32 * half);            // of P
        const uint32_t to = tmem_addr(tb, quad * 32, T_O + 128 * t + (D / 2) * half);      // and of O
        const float sl2 = P.scale_log2;
        float m_ref = -INFINITY, l_sum = 0.f;
        if (t == 0 || two) {
            for (int j = 0; j < tiles; ++j) {
                wait(&bar_s[t], j & 1, 7);
                __syncwarp();
                tc_fence_after();
                float x[2][32];
                if (warp_live) {
                    tmem_ld32(ts, x[0]);
                    tmem_ld32(ts + 32, x[1]);
                    tmem_wait_ld();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_r[t]);           // S may be overwritten
                // P V of the tile before is done: P may be overwritten, O rescaled
                bool waited = j == 0;
                auto free = [&] {
                    if (!waited) {
                        wait(&bar_o[t], (j - 1) & 1, 8);
                        __syncwarp();
                        tc_fence_after();
                        waited = true;
                    }
                };
                if (warp_live) {
                    const int hi = sees - (w.t0 + j) * kTile - 64 * half;      // this half's columns [0, hi) are visible
                    if (hi < 64) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[c][e] = 32 * c + e < hi ? x[c][e] : -INFINITY;
                    }
                    // P = 2^(s - m) with the reference max of the tiles before, while the tile's own max is
                    // taken beside it (it would wait for itself in a pass of its own).  Only if that max
                    // passes the reference by more than the margin is m moved, O and l rescaled and P taken
                    // again, which is rare.  The rows' two warps decide together.
                    float ls;
                    if (j == 0) {              // no reference yet: the row's max first, through its two threads
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 64; e += 2) mx[e / 2 & 3] = fmaxf(mx[e / 2 & 3], fmaxf(x[e / 32][e % 32], x[e / 32][e % 32 + 1]));
                        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                        if (half == 0) s_pair[r] = mt;
                        asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                        if (half == 1) s_pair[r] = mt = fmaxf(mt, s_pair[r]);
                        asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                        m_ref = s_pair[r];
                    }
                    while (true) {
                        float mt;
                        softmax_half(x, sl2, m_ref, tp, ls, mt, free);
                        if (!bar_sync_or(pair, 64, mt > m_ref + kMargin)) break;
                        if (half == 0) s_pair[r] = mt;
                        asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                        if (half == 1) s_pair[r] = mt = fmaxf(mt, s_pair[r]);
                        asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                        mt = s_pair[r];
                        const bool up = mt > m_ref + kMargin;
                        const float alpha = !up ? 1.f : m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - mt);
                        if (up) m_ref = mt;
                        l_sum *= alpha;
                        tmem_wait_st();
                        if (j > 0) {
#pragma unroll 1
                            for (int c0 = 0; c0 < D / 2; c0 += 32) {
                                float o[32];
                                tmem_ld32(to + c0, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= alpha;
                                tmem_st32(to + c0, o);
                            }
                        }
                    }
                    l_sum += ls;
                    tmem_wait_st();
                } else {
                    free();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_p[t]);
            }
            wait(&bar_o[t], (tiles - 1) & 1, 10);
            __syncwarp();
            if (warp_live && !bar_sync_or(pair, 64, stopped())) {
                tc_fence_after();
                if (half == 1) s_pair[r] = l_sum;
                asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                const int64_t row = live ? row_of(P, w.hk, w.row0 + r) : 0;
                if (live && half == 0) {
                    l_sum += s_pair[r];
                    if (m_ref == -INFINITY && l_sum != 0.f) m_ref = 0.f;       // every visible score is NaN: so is the row
                    ml[row] = make_float2(m_ref, l_sum);
                }
                // O leaves row by row through shared memory (a lane holds a row: 32 rows at once would be 32
                // partial lines per store), in the space of this row tile's queries, whose products are done.  It
                // holds 64 columns of the tile: one half after the other at d = 128.
                constexpr int kC = D / 8;                        // 16-byte chunks of half a row, chunk c at c ^ (row & 7)
                float4 *st = reinterpret_cast<float4 *>(sm_q + t * kTileBytes) + quad * 32 * kC;
                const int rows = min(32, w.nrows - (t * kTile + quad * 32));
                for (int h = 0; h < 2; ++h) {
                    if (half == h) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D / 2; c0 += 32) {
                            float o[32];
                            tmem_ld32(to + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                st[lane * kC + (((c0 + e) / 4) ^ (lane & 7))] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    }
                    asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
#pragma unroll 4
                    for (int i0 = half * 32; i0 < rows * kC; i0 += 64) {
                        const int i = i0 + lane, rr = min(i / kC, 31), c = i % kC;
                        const int64_t dst = __shfl_sync(0xffffffffu, row, rr);
                        if (i < rows * kC)
                            reinterpret_cast<float4 *>(P.part_o + (w.part * P.rows + dst) * D + (D / 2) * h)[c] = st[rr * kC + (c ^ (rr & 7))];
                    }
                    asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) tmem_dealloc(tb, 512);
    if (tid == 0) P.item_status[item] = s_status;
    grid_end();
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

// Tiles on their way: at d = 128 three CTAs an SM of two tiles (64 KB each, at most 136 registers a thread, of which 16 rows
// spill 16 bytes) beat two CTAs of three, because one CTA's start lies behind two others' loads (own keys of 64 requests of
// up to 1024 tokens, 32 query heads on 8, 35 against 40 us; of 32 requests with 4 tokens each, 47 against 61 us, both with
// the splits of that time; with the present ones 33 and 41 us).  One set of CTAs that stay and take one item after the
// other without a gap in the loads was slower (37 and 55 us): the gaps of one CTA lie behind the others anyway.
template <int D, int NT>
constexpr int warp_stages() { return D == 128 ? 2 : 3; }
template <int D, int NT>
constexpr int warp_smem() { return warp_stages<D, NT>() * 2 * kWKeys * D * 2 + 1024; }

// NT: column tiles of 8 rows.  TW: as above.
template <int D, int NT, bool TW>
__global__ void __maxnreg__(136)
gdn_warp_attn_kernel(const __grid_constant__ PrefixParams P, const __grid_constant__ PrefixMaps M) {
    constexpr int kHalves = D / 64;
    constexpr int kHalfBytes = kWKeys * 128;
    constexpr int kWStages = warp_stages<D, NT>();
    constexpr int kTileBytes = kHalves * kHalfBytes;          // of K, and of V
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kWStages], empty[kWStages];
    __shared__ float2 s_ml[4][kWRows];
    __shared__ int s_abort, s_status;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int item = P.first_item + blockIdx.x;
    if (P.first_item == 0) grid_wait();
    grid_next();
    if (item == 0 && tid == 0) P.ws->status = P.ws->timeout_where = 0;
    const Item w = item_of<kWKeys, kWRows, kWMinTiles>(P, item);
    const int tiles = w.t1 - w.t0;
    float2 *ml = P.part_ml + w.part * P.rows;
    if (tiles == 0) {                          // an empty part: nothing visible
        if (tid < w.nrows) ml[row_of(P, w.hk, w.row0 + tid)] = make_float2(-INFINITY, 0.f);
        if (tid == 0) P.item_status[item] = 0;
        grid_end();
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kWStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 4);
        }
        fence_mbar_init();
        s_abort = s_status = 0;
    }
    __syncthreads();

    // Bounded wait; one that gives up marks the CTA as stopping, and every further one gives up at once: the loads
    // stop, the other warps run through their tiles (on unspecified data).
    auto stopped = [&] { return *reinterpret_cast<volatile int *>(&s_abort) != 0; };
    auto wait = [&](uint64_t *bar, uint32_t parity, int where) {
        if constexpr (TW) {
            if (stopped() || mbar_poll(bar, parity, P.wait_iters)) return;
        } else {
            if (mbar_try_wait(bar, parity)) return;
            for (uint32_t it = 0; it < kPWaitIters / 16; ++it) {
                if (mbar_wait_some(bar, parity)) return;
                if (stopped()) return;
            }
        }
        if (atomicExch(&s_abort, 1) == 0) atomicOr(&s_status, (int)GDN_ERR_TIMEOUT | where << 16);
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
                else atomicOr(&s_status, (int)GDN_ERR_INVALID_ARG);
            }
            if (issued >= kWStages) {
                wait(&empty[slot], (issued / kWStages - 1) & 1, 11);
                __syncwarp();
                if (__any_sync(0xffffffffu, stopped())) break;     // the slot may still be in use
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2 * kTileBytes);
            __syncwarp();
            if (mine)
                tma_load_3d(sm + (2 * slot + value) * kTileBytes + half * kHalfBytes + box * box_rows * 128,
                            value ? &M.v : &M.k, &full[slot], half * 64, w.hk, row);
            __syncwarp();
        }
        if (__any_sync(0xffffffffu, stopped()) && lane == 0)       // gave up: the loads in flight still land
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
        const int newest = (w.n >= 0 && P.causal) ? w.keys - (P.L - 1) : w.keys;     // keys before it are for every row
        // ldmatrix addresses inside this warp's 16 rows: K (row, 8 columns), V transposed
        const int krow = warp * 16 + (lane & 15), kchunk = lane >> 4;
        const int vrow = warp * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, vchunk = (lane >> 3) & 1;
        const uint32_t smb = smem_u32(sm);
        for (int i = 0; i < tiles; ++i) {
            const int slot = i % kWStages;
            wait(&full[slot], (i / kWStages) & 1, 12);
            __syncwarp();
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
                const int last = min(16, w.keys - key0);
                if (last < 16 || newest < key0 + 16) {             // not every key is for every row
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key0 + (lane >> 2) + (e >> 1) * 8 >= sees[n][e & 1]) s[n][e] = -INFINITY;
                    // nor is every V row (see the file comment)
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
                    if (found) atomicOr(&s_status, kItemNonfinite);
                    fence_async_smem();        // before the slot's next load
                    __syncwarp();
                }
                // The reference max moves only when a score passes it by more than the margin: a vote, and
                // the rows' maxima across lanes only then
                bool up = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) up = up || s[n][e] * sl2 > m_ref[n][e & 1] + kMargin;
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mt = fmaxf(s[n][e], s[n][e + 2]) * sl2;
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                            if (mt > m_ref[n][e] + kMargin) {
                                const float alpha = m_ref[n][e] == -INFINITY ? 0.f : ex2_approx(m_ref[n][e] - mt);
                                m_ref[n][e] = mt;
                                l_sum[n][e] *= alpha;
#pragma unroll
                                for (int d0 = 0; d0 < D / 16; ++d0) {
                                    acc[d0][n][e] *= alpha;
                                    acc[d0][n][e + 2] *= alpha;
                                }
                            }
                        }
                }
                uint32_t pf[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mu = m_ref[n][e] == -INFINITY ? 0.f : m_ref[n][e];
                        s[n][e] = ex2_approx(fmaf(s[n][e], sl2, -mu));
                        s[n][e + 2] = ex2_approx(fmaf(s[n][e + 2], sl2, -mu));
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
    // The ring is free: the warps' O^T go there, [warp][row][d], with 4 floats behind a row (a warp's writes to its 4
    // rows x 8 columns then meet no bank twice)
    constexpr int kRow = D + 4;
    static_assert(4 * NT * 8 * kRow * 4 <= kWStages * 2 * kTileBytes, "the warps' O must fit the ring");
    __syncthreads();
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
                float *dst = so + (warp * (NT * 8) + row) * kRow + (lane >> 2);
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
            const float4 u = reinterpret_cast<const float4 *>(so)[(y * (NT * 8) + row) * (kRow / 4) + c];
            o.x += u.x, o.y += u.y, o.z += u.z, o.w += u.w;
        }
        reinterpret_cast<float4 *>(P.part_o + (w.part * P.rows + row_of(P, w.hk, w.row0 + row)) * D)[c] = o;
    }
    if (tid == 0) P.item_status[item] = s_status;
    grid_end();
}

// The item that made part `p` of row (n, l, h).
__device__ __forceinline__ int64_t item_at(const PrefixParams &P, int p, int n, int l, int h) {
    const int hk = h / P.G, in_seq = l * P.G + (h - hk * P.G);
    if (p < P.prefix_splits)
        return ((int64_t)hk * P.prefix_splits + p) * P.prefix_tiles + ((int64_t)n * P.L * P.G + in_seq) / P.prefix_rows;
    return P.items_of_prefix +
           (((int64_t)n * P.own_splits + (p - P.prefix_splits)) * P.Hkv + hk) * P.own_tiles + in_seq / P.own_rows;
}

// One warp per row (n, l, h): lane holds D / 32 columns.  A lane first takes the (m, l) of parts of its own, so
// that the parts' rows are read without waiting for one another.
template <int D>
__global__ void __launch_bounds__(128) gdn_attn_combine_kernel(const __grid_constant__ PrefixParams P, int parts) {
    constexpr int C = D / 32;
    const int64_t row = ((int64_t)blockIdx.x * 128 + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int h = (int)(row % P.H), l = (int)(row / P.H % P.L), n = (int)(row / P.H / P.L);
    const int s = row < P.rows ? own_len(P, n) : 0;       // an input: on its way beside the wait
    grid_wait();
    if (row >= P.rows) return;
    float m = -INFINITY, sum = 0.f, acc[C];
    int status = s < 0 ? (int)GDN_ERR_INVALID_ARG : 0;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    for (int p0 = 0; p0 < parts; p0 += 32) {       // 32 parts at a time, joined to what came before
        float2 a = make_float2(-INFINITY, 0.f);
        if (p0 + lane < parts) {
            a = P.part_ml[(p0 + lane) * P.rows + row];
            status |= P.item_status[item_at(P, p0 + lane, n, l, h)];
        }
        float top = a.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, m);
        if (top == -INFINITY) continue;
        const float back = m == -INFINITY ? 0.f : ex2_approx(m - top);
        m = top;
        const float f = a.x == -INFINITY ? 0.f : ex2_approx(a.x - top);
        float part = a.x == -INFINITY ? 0.f : f * a.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        sum = sum * back + part;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] *= back;
        uint32_t some = __ballot_sync(0xffffffffu, a.x != -INFINITY);     // parts that see a key
        while (some) {
            float x[4][C], g[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {          // four rows on their way at a time
                const int p = some ? __ffs(some) - 1 : -1;
                some &= some - 1;
                g[i] = __shfl_sync(0xffffffffu, f, max(p, 0));
                if (p < 0) g[i] = 0.f;
#pragma unroll
                for (int c = 0; c < C; ++c) x[i][c] = 0.f;
                if (p >= 0) {
                    const float *o = P.part_o + ((p0 + p) * P.rows + row) * D + lane * C;
                    if constexpr (C == 4) {
                        const float4 u = *reinterpret_cast<const float4 *>(o);
                        x[i][0] = u.x, x[i][1] = u.y, x[i][2] = u.z, x[i][3] = u.w;
                    } else {
                        const float2 u = *reinterpret_cast<const float2 *>(o);
                        x[i][0] = u.x, x[i][1] = u.y;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < C; ++c) acc[c] = fmaf(g[i], x[i][c], acc[c]);
        }
    }
    status = __reduce_or_sync(0xffffffffu, status);
    if (status) {
        if (lane == 0 && (status & 0xff)) {
            if ((status & 0xff) == GDN_ERR_INVALID_ARG) {
                atomicCAS(&P.ws->status, 0, (int)GDN_ERR_INVALID_ARG);
            } else {                               // a wait gave up somewhere (perhaps beside bad pages)
                atomicExch(&P.ws->status, (int)GDN_ERR_TIMEOUT);
                atomicExch(&P.ws->timeout_where, status >> 16);
            }
        }
        if (s < 0) return;
    }
    if (m != -INFINITY) {
        const float inv = 1.f / sum;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] *= inv;
        if (status & kItemNonfinite) {             // set to zero in the product: they reach the rows that see them
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
    } else if (P.prefix > 0 || (P.causal ? s - (P.L - 1 - l) : s) > 0) {      // keys, but every score is -inf: 0 / 0
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = NAN;
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
           (D->scale == 0.f || (D->scale > 0.f && std::isfinite(1.5f * D->scale))) && D->num_heads % D->num_kv_heads == 0 &&
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
    size_t off_status, off_ml, off_o, bytes;
};

// Splits of `tiles` key tiles over `base` equal lists for gdn_tile_attn_kernel, beside other work of `beside`
// SM-microseconds in the same call.  A CTA has an SM to itself and takes kTileUs a key tile and kStartUs for its start and
// end (measured at two row tiles, d = 128; taken for d = 64 and for one row tile too, where a tile is about half and
// a quarter of that work); the call takes as long as its waves of CTAs, or as all its work on all
// SMs, and each part a little in the combine step.  With own keys beside it a prefix is thus cut into fewer
// parts than would fill the GPU: 16384 keys for 256 requests of up to 512 own tokens, 3 parts of 32 CTAs
// 108 us, 4 parts 122 us (2 parts 131 us); the prefix alone, 92 us and 74 us.
// The host knows the tables' room, not the lengths, so the prefix's own time may grow by a third and 6.5 us at the most: 64
// requests of up to 1024 own tokens over 8192 prefix keys take 45 us with tables of that room (6 parts; 5 parts 48 us,
// 8 parts 50) and with 32 times it (150 us without the limit); 24 x 8 drafts at d = 64 over 1001 keys 41 us (1 part; 2 parts 44).
int tile_split(int64_t base, int64_t tiles, double beside) {
    constexpr double kTileUs = 1.6, kStartUs = 12.0, kPartUs = 0.3, kMost = 1.35, kMostUs = 6.5;
    int best = 1;
    double least = 1e300, cost = 1e300;
    for (int pass = 0; pass < 2; ++pass)
        for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
            const double cta = (double)((tiles + s - 1) / s) * kTileUs + kStartUs;
            const double waves = (double)((base * s + kSms - 1) / kSms) * cta;
            if (pass == 0) {
                least = std::min(least, waves);
                continue;
            }
            if (waves > kMost * least + kMostUs) continue;
            const double c = std::max(waves, ((double)(base * s) * cta + beside) / kSms) + kPartUs * s;
            if (c < cost * 0.999) cost = c, best = s;
        }
    return best;
}

// The same for gdn_warp_attn_kernel, whose CTAs share an SM and whose lists differ in length: about two CTAs for
// each of its places on the GPU while no split gets shorter than its least.  A part costs its rows of O a write and a
// read: 64 requests of up to 1024 own tokens over 8192 prefix keys take 45.7 us with 6 CTAs a SM (2 parts) and 48.9 with
// 8 (3 parts), 32 blocks of 4 over 32768 104 and 110 us; with 4 CTAs a SM, 32 requests of up to 16384 own
// tokens wait for the longest (194 against 187 us).
int warp_split(int64_t base, int64_t keys) {
    const int64_t most = (keys + kWKeys * kWMinTiles - 1) / (kWKeys * kWMinTiles);
    return (int)std::max<int64_t>(1, std::min<int64_t>({(6 * kSms + base - 1) / base, most, kMaxSplits}));
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
    p.own_splits = !own_room ? 0 : p.own_warp ? warp_split(own_base, own_room) : tile_split(own_base, (own_room + kTile - 1) / kTile, 0.0);
    // Own keys beside the prefix: half of the tables' room at 6.4 TB/s, but not above 1024 tokens a sequence (tables with
    // room for more are mostly as wide as a sequence may ever get), and 1.7 SM-microseconds a CTA for its start and end.
    const double own_us = (double)D->num_seqs * std::min<int64_t>(own_room / 2, 1024) * D->num_kv_heads * D->head_dim * 4 / 6.4e6 * kSms +
                          1.7 * (double)(own_base * p.own_splits);
    p.prefix_splits = !D->prefix_len ? 0 : p.prefix_warp ? warp_split(prefix_base, D->prefix_len)
                                                         : tile_split(prefix_base, ((int64_t)D->prefix_len + kTile - 1) / kTile, own_us);
    p.prefix_items = (int64_t)D->num_kv_heads * p.prefix_tiles * p.prefix_splits;
    p.own_items = (int64_t)D->num_seqs * D->num_kv_heads * p.own_tiles * p.own_splits;
    p.parts = p.prefix_splits + p.own_splits;
    p.off_status = sizeof(WorkspaceHeader);
    p.off_ml = p.off_status + round256((size_t)(p.prefix_items + p.own_items) * 4);
    p.off_o = p.off_ml + round256((size_t)p.parts * p.rows * 8);
    p.bytes = p.off_o + round256((size_t)p.parts * p.rows * D->head_dim * 4);
    return p;
}

template <int D>
constexpr int tile_smem() { return (2 + kStages) * kTile * D * 2 + 1024; }

// Raises the kernels' dynamic shared memory limits, once per device.
template <int D, bool TW>
cudaError_t prepare_device() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    e = cudaFuncSetAttribute(gdn_tile_attn_kernel<D, TW>, attr, tile_smem<D>());
    // the shares that its warps take add up to what it is launched with, or they would wait for ever
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, gdn_tile_attn_kernel<D, TW>);
    if (e == cudaSuccess && fa.numRegs < kRegsLaunch) e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_warp_attn_kernel<D, 1, TW>, attr, warp_smem<D, 1>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_warp_attn_kernel<D, 2, TW>, attr, warp_smem<D, 2>());
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// A launch that may overlap the kernel before it (see grid_wait).
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                             const Args &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// One launch over items [first, first + count).
template <int D, bool TW>
cudaError_t launch_parts(PrefixParams P, const PrefixMaps &maps, bool warp, int64_t rows, int64_t first, int64_t count,
                         cudaStream_t st) {
    if (count == 0) return cudaSuccess;
    P.first_item = (int32_t)first;
    if (!warp) return launch_dependent(gdn_tile_attn_kernel<D, TW>, (unsigned)count, kTThreads, tile_smem<D>(), st, P, maps);
    if (rows <= 8) return launch_dependent(gdn_warp_attn_kernel<D, 1, TW>, (unsigned)count, kWThreads, warp_smem<D, 1>(), st, P, maps);
    return launch_dependent(gdn_warp_attn_kernel<D, 2, TW>, (unsigned)count, kWThreads, warp_smem<D, 2>(), st, P, maps);
}

template <int D, bool TW>
gdn_status launch(const PrefixParams &P, const PrefixMaps &maps, const Plan &plan, cudaStream_t st) {
    if (prepare_device<D, TW>() != cudaSuccess) return GDN_ERR_CUDA;
    const int64_t own_rows = (int64_t)P.L * P.G, all_rows = P.N * own_rows;
    const bool both = plan.prefix_warp == plan.own_warp && plan.own_items > 0;
    cudaError_t e = cudaSuccess;
    if (plan.prefix_items + plan.own_items == 0) e = cudaMemsetAsync(P.ws, 0, sizeof(WorkspaceHeader), st);
    if (e == cudaSuccess)
        e = launch_parts<D, TW>(P, maps, plan.prefix_warp, plan.prefix_items ? all_rows : own_rows, 0,
                            plan.prefix_items + (both ? plan.own_items : 0), st);
    if (e == cudaSuccess && !both) e = launch_parts<D, TW>(P, maps, plan.own_warp, own_rows, plan.prefix_items, plan.own_items, st);
    if (e == cudaSuccess)
        e = launch_dependent(gdn_attn_combine_kernel<D>, (unsigned)((plan.rows + 3) / 4), 128, 0, st, P, plan.parts);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" size_t gdn_prefix_attn_workspace_size(const gdn_prefix_attn_desc *desc) {
    if (!desc_ok(desc) || !desc_supported(desc)) return 0;
    return plan_of(desc).bytes;
}

// wait_iters 0: the normal bound.
static gdn_status prefix_attn(const gdn_prefix_attn_desc *D, const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *prefix_pages, const int32_t *block_table, const int32_t *seq_lens, void *out,
                              void *workspace, size_t workspace_bytes, uint32_t wait_iters, gdn_stream_t stream) {
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
    struct Span {
        uintptr_t lo, hi;
        Span(const void *p, size_t n) : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + (p ? n : 0)) {}
        bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
    };
    const size_t cache = (size_t)D->num_pages * D->page_size * D->num_kv_heads * D->head_dim * 2;
    const size_t io = (size_t)plan.rows * D->head_dim * 2;
    const Span written[] = {{out, io}, {workspace, plan.bytes}};
    const Span read[] = {{q, io}, {k_cache, cache}, {v_cache, cache},
                         {prefix_pages, ((size_t)D->prefix_len + D->page_size - 1) / D->page_size * 4},
                         {block_table, (size_t)D->num_seqs * D->table_width * 4}, {seq_lens, (size_t)D->num_seqs * 4}};
    if (written[0].meets(written[1])) return GDN_ERR_INVALID_ARG;
    for (const Span &o : written)
        for (const Span &i : read)
            if (o.meets(i)) return GDN_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    PrefixParams P = {};
    P.q = static_cast<const __nv_bfloat16 *>(q);
    P.v_cache = static_cast<const __nv_bfloat16 *>(v_cache);
    P.out = static_cast<__nv_bfloat16 *>(out);
    P.prefix_pages = prefix_pages, P.block_table = block_table, P.seq_lens = seq_lens;
    P.ws = reinterpret_cast<WorkspaceHeader *>(ws);
    P.item_status = reinterpret_cast<int32_t *>(ws + plan.off_status);
    P.part_ml = reinterpret_cast<float2 *>(ws + plan.off_ml);
    P.part_o = reinterpret_cast<float *>(ws + plan.off_o);
    P.rows = plan.rows;
    P.N = D->num_seqs, P.L = D->num_tokens, P.H = D->num_heads, P.Hkv = D->num_kv_heads, P.G = P.H / P.Hkv;
    P.W = D->table_width, P.page = D->page_size, P.pages = D->num_pages, P.prefix = D->prefix_len, P.causal = D->causal;
    P.items_of_prefix = (int32_t)plan.prefix_items, P.prefix_tiles = plan.prefix_tiles, P.prefix_splits = plan.prefix_splits;
    P.prefix_rows = plan.prefix_warp ? kWRows : kRows, P.own_rows = plan.own_warp ? kWRows : kRows;
    P.own_tiles = plan.own_tiles, P.own_splits = plan.own_splits;
    const double scale = D->scale > 0.f ? D->scale : 1.0 / std::sqrt((double)D->head_dim);
    P.scale_log2 = (float)(1.4426950408889634 * scale);
    PrefixMaps maps;
    if (!cache_map(&maps.k, k_cache, D) || !cache_map(&maps.v, v_cache, D)) return GDN_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    P.wait_iters = wait_iters;
    if (wait_iters) return D->head_dim == 64 ? launch<64, true>(P, maps, plan, st) : launch<128, true>(P, maps, plan, st);
    return D->head_dim == 64 ? launch<64, false>(P, maps, plan, st) : launch<128, false>(P, maps, plan, st);
}

extern "C" gdn_status gdn_prefix_attn(const gdn_prefix_attn_desc *desc, const void *q, const void *k_cache,
                                      const void *v_cache, const int32_t *prefix_pages, const int32_t *block_table,
                                      const int32_t *seq_lens, void *out, void *workspace, size_t workspace_bytes,
                                      gdn_stream_t stream) {
    return prefix_attn(desc, q, k_cache, v_cache, prefix_pages, block_table, seq_lens, out, workspace, workspace_bytes, 0,
                       stream);
}

extern "C" gdn_status gdn_prefix_attn_test_wait_limit(const gdn_prefix_attn_desc *desc, const void *q, const void *k_cache,
                                                      const void *v_cache, const int32_t *prefix_pages,
                                                      const int32_t *block_table, const int32_t *seq_lens, void *out,
                                                      void *workspace, size_t workspace_bytes, uint32_t wait_iters,
                                                      gdn_stream_t stream) {
    if (wait_iters == 0) return GDN_ERR_INVALID_ARG;
    return prefix_attn(desc, q, k_cache, v_cache, prefix_pages, block_table, seq_lens, out, workspace, workspace_bytes,
                       wait_iters, stream);
}
