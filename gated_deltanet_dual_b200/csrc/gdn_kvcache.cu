// gdn_kvcache.cu -- block tables, slots and positions of a serving step's new tokens
// (gdn_kv_extend of include/gdn_kvcache.h).
//
// Two exclusive sums over the sequences -- pages needed and tokens -- decide everything: which entry of the
// free list a new page takes and which packed row a token has.  A few kilobytes are read and 8 bytes per token
// written, so the call is bound by latency: one launch, in which every CTA runs the whole scan itself (four
// sequences per thread and pass; the lengths come from L2) and then writes only its own range of token
// rows.  A token whose index starts a page also writes that page's table entry, so entries have one writer and
// no CTA reads an entry that another one writes (rows on new pages take the page from the free list).  One
// decode step of 64 sequences takes 5.5 us, a step of 1024 sequences with up to 256 new tokens each 8.2 us, where an
// empty kernel takes about 2: a chain of three dependent reads (lengths, page, entry) between two barriers.
#include <algorithm>
#include <climits>

#include "gdn_internal.cuh"
#include "../../include/gdn_kvcache.h"

namespace gdn {
namespace {

constexpr int kXItems = 4;                      // sequences per thread and pass
constexpr int kXRows = 4096;                    // most token rows of a CTA
constexpr int kXDirect = 4;                     // a thread writes so many of its sequence's rows by itself
constexpr int kXWide = 64;                      // longer runs are for the whole CTA, shorter ones for a warp
constexpr int kXList = kXRows / (kXDirect + 1) + 2;

struct ExtendParams {
    int32_t *table;
    const int32_t *lens, *fresh, *free_pages, *free_count;
    int32_t *slot_map, *positions, *cu, *lens_out, *free_left, *status;
    int32_t N, W, page, shift, F, M, prefix, rows_per_cta;    // shift: page = 2^shift, or -1
};

// x / page for 0 <= x < 2^32
__device__ __forceinline__ uint32_t pages_in(const ExtendParams &P, uint32_t x) {
    return P.shift >= 0 ? x >> P.shift : x / (uint32_t)P.page;
}

// One sequence's rows.
struct Run {
    int64_t cu, page0;          // its first row; the pages taken before its own
    int32_t n, len, have;       // own tokens, pages it had
    int32_t lo, hi;             // rows [lo, hi) of this CTA's range that are its own
    bool refused;
};

__device__ __forceinline__ void write_row(const ExtendParams &P, const Run &r, int row, int top) {
    if (r.refused) {
        P.slot_map[row] = -1;
        P.positions[row] = -1;
        return;
    }
    const int i = r.len + (int)(row - r.cu);
    const int j = (int)pages_in(P, i), off = i - j * P.page;
    int64_t page;
    int32_t *entry = P.table + (int64_t)r.n * P.W + j;
    if (j < r.have) {
        page = *entry;
    } else {
        page = P.free_pages[top - 1 - (r.page0 + (j - r.have))];
        if (off == 0) *entry = (int32_t)page;
    }
    // an entry that no cache can hold must not turn into a slot of another page
    int64_t slot = page * P.page + off;
    if (page < 0 || slot > INT32_MAX) {
        slot = -1;
        if (P.status) atomicExch(P.status, (int32_t)GDN_ERR_INVALID_ARG);
    }
    P.slot_map[row] = (int32_t)slot;
    P.positions[row] = (int32_t)min((int64_t)P.prefix + i, (int64_t)INT32_MAX);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) gdn_kv_extend_kernel(const __grid_constant__ ExtendParams P) {
    constexpr int kWarps = THREADS / 32;
    __shared__ int64_t s_new[2][32], s_need[2][32];     // the warps' sums, of even and odd passes
    __shared__ Run s_list[kXList];
    __shared__ int s_count;
    __shared__ unsigned long long s_taken;      // pages that served sequences take
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = (int)min((int64_t)blockIdx.x * P.rows_per_cta, (int64_t)P.M);
    const int row1 = (int)min((int64_t)row0 + P.rows_per_cta, (int64_t)P.M);
    const int32_t count = *P.free_count;
    const int64_t room = min((int64_t)P.W * P.page, (int64_t)INT32_MAX);     // lengths are int32
    bool bad = false;
    int64_t need_before = 0, new_before = 0;    // sums of the earlier passes
    if (tid == 0) s_taken = 0, s_count = 0;

    for (int64_t base = 0, pass = 0; base < P.N; base += THREADS * kXItems, ++pass) {
        const int par = (int)(pass & 1);
        int32_t len[kXItems], w[kXItems], have[kXItems], need[kXItems];
        bool wrong[kXItems];
        int64_t my_need = 0, my_new = 0;
        const int64_t n0 = base + tid * kXItems;
#pragma unroll
        for (int i = 0; i < kXItems; ++i) {
            const bool in = n0 + i < P.N;
            len[i] = in ? P.lens[n0 + i] : 0;
            w[i] = in ? P.fresh[n0 + i] : 0;
        }
#pragma unroll
        for (int i = 0; i < kXItems; ++i) {
            wrong[i] = len[i] < 0 || w[i] < 0 || (int64_t)len[i] + w[i] > room;
            w[i] = max(w[i], 0);
            my_new += w[i];
            // lengths with their new tokens stay below 2^31 (room), pages too: sums below 2^32
            have[i] = wrong[i] ? 0 : (int)pages_in(P, (uint32_t)len[i] + (uint32_t)(P.page - 1));
            need[i] = wrong[i] ? 0 : (int)pages_in(P, (uint32_t)len[i] + (uint32_t)w[i] + (uint32_t)(P.page - 1)) - have[i];
            my_need += need[i];
        }
        // Both sums in one scan.  A sequence whose rows pass M is refused and takes no pages; as the rows' sum only
        // grows, so is every sequence behind it, and counting its pages changes nothing for the others.
        int64_t x = my_new, y = my_need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) x += a, y += b;
        }
        if (lane == 31) s_new[par][warp] = x, s_need[par][warp] = y;
        __syncthreads();
        int64_t cu = new_before + x - my_new, before = need_before + y - my_need;
        {                                       // the warps before this one, and all of them
            int64_t a = lane < kWarps ? s_new[par][lane] : 0, b = lane < kWarps ? s_need[par][lane] : 0;
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1) {
                const int64_t c = __shfl_up_sync(0xffffffffu, a, o), d = __shfl_up_sync(0xffffffffu, b, o);
                if (lane >= o) a += c, b += d;
            }
            const int64_t pa = __shfl_sync(0xffffffffu, a, max(warp - 1, 0)), pb = __shfl_sync(0xffffffffu, b, max(warp - 1, 0));
            if (warp > 0) cu += pa, before += pb;
            new_before += __shfl_sync(0xffffffffu, a, kWarps - 1);
            need_before += __shfl_sync(0xffffffffu, b, kWarps - 1);
        }
        const int top = min(max(count, 0), P.F);
        const bool writer = pass % gridDim.x == blockIdx.x;     // this pass's per-sequence outputs
        bool listed = false;
#pragma unroll
        for (int i = 0; i < kXItems; ++i) {
            const int64_t n = n0 + i;
            if (n < P.N) {
                Run r;
                r.cu = cu, r.page0 = before, r.n = (int32_t)n, r.len = len[i], r.have = have[i];
                r.refused = wrong[i] || cu + w[i] > P.M || (need[i] > 0 && before + need[i] > top);
                r.lo = (int)min(max(cu, (int64_t)row0), (int64_t)row1);
                r.hi = (int)min(cu + w[i], (int64_t)row1);
                if (r.refused) bad = true;
                else if (need[i] > 0) atomicMax(&s_taken, (unsigned long long)(before + need[i]));
                if (writer) {
                    P.cu[n] = (int32_t)min(cu, (int64_t)INT32_MAX);
                    P.lens_out[n] = r.refused ? len[i] : len[i] + w[i];
                }
                if (r.hi - r.lo > kXDirect) {
                    s_list[atomicAdd(&s_count, 1)] = r;
                    listed = true;
                } else {
                    for (int row = r.lo; row < r.hi; ++row) write_row(P, r, row, top);
                }
                cu += w[i];
                before += need[i];
            }
        }
        if (__syncthreads_or(listed)) {
            const int runs = s_count;
            for (int e = warp; e < runs; e += kWarps) {                     // short runs: a warp each
                const Run r = s_list[e];
                if (r.hi - r.lo <= kXWide)
                    for (int row = r.lo + lane; row < r.hi; row += 32) write_row(P, r, row, top);
            }
            for (int e = 0; e < runs; ++e) {                                // long ones: the CTA
                if (s_list[e].hi - s_list[e].lo <= kXWide) continue;
                const Run r = s_list[e];
                for (int row = r.lo + tid; row < r.hi; row += THREADS) write_row(P, r, row, top);
            }
            __syncthreads();
            if (tid == 0) s_count = 0;          // the next pass's barrier comes before its first run
        }
    }
    for (int64_t row = max(new_before, (int64_t)row0) + tid; row < row1; row += THREADS) {     // padding rows
        P.slot_map[row] = -1;
        P.positions[row] = -1;
    }
    if (blockIdx.x == 0) {
        const int top = min(max(count, 0), P.F);
        if (tid == 0) {                         // the last pass's barrier came after every atomicMax
            P.cu[P.N] = (int32_t)min(new_before, (int64_t)INT32_MAX);
            *P.free_left = top - (int)s_taken;
        }
        if ((bad || top != count) && P.status) atomicExch(P.status, (int32_t)GDN_ERR_INVALID_ARG);
    }
}

struct Span {
    uintptr_t lo, hi;
    Span(const void *p, int64_t n) : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + (p ? 4 * (uintptr_t)n : 0)) {}
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_kv_extend(const gdn_kv_extend_desc *D, int32_t *block_table, const int32_t *seq_lens,
                                    const int32_t *new_lens, const int32_t *free_pages, const int32_t *free_count,
                                    int32_t *slot_map, int32_t *positions, int32_t *cu_new, int32_t *seq_lens_out,
                                    int32_t *free_left, int32_t *device_status, gdn_stream_t stream) {
    if (!D || D->num_seqs < 1 || D->table_width < 1 || D->page_size < 1 || D->num_free < 0 || D->max_new_tokens < 0 ||
        D->prefix_len < 0 || D->reserved[0] || D->reserved[1] || D->num_seqs > INT32_MAX - 8192)
        return GDN_ERR_INVALID_ARG;
    if (!block_table || !seq_lens || !new_lens || !free_count || !cu_new || !seq_lens_out || !free_left ||
        (D->num_free > 0 && !free_pages) || (D->max_new_tokens > 0 && (!slot_map || !positions)))
        return GDN_ERR_INVALID_ARG;
    const void *all[] = {block_table, seq_lens, new_lens, free_pages, free_count, slot_map, positions, cu_new,
                         seq_lens_out, free_left, device_status};
    for (const void *p : all)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return GDN_ERR_ALIGNMENT;
    const int64_t N = D->num_seqs, M = D->max_new_tokens;
    const Span in[] = {{seq_lens, N}, {new_lens, N}, {free_pages, D->num_free}, {free_count, 1}};
    const Span out[] = {{block_table, N * D->table_width}, {slot_map, M}, {positions, M}, {cu_new, N + 1},
                        {seq_lens_out, N}, {free_left, 1}, {device_status, 1}};
    for (const Span &o : out) {
        for (const Span &i : in)
            if (o.meets(i)) return GDN_ERR_INVALID_ARG;
        for (const Span &p : out)
            if (&p != &o && o.meets(p)) return GDN_ERR_INVALID_ARG;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (device_status && cudaMemsetAsync(device_status, 0, sizeof(int32_t), st) != cudaSuccess) return GDN_ERR_CUDA;
    int shift = -1;
    if ((D->page_size & (D->page_size - 1)) == 0)
        for (shift = 0; (1 << shift) < D->page_size;) ++shift;
    // Small CTAs while one pass of them covers the sequences (their barriers are cheaper), large ones for fewer
    // passes after that; a row per thread, more only when that would pass two CTAs per SM.
    const int threads = N <= 256 * kXItems ? 256 : 1024;
    const int32_t rows = (int32_t)std::min<int64_t>(kXRows, std::max<int64_t>(threads, (M + 295) / 296));
    const ExtendParams P = {block_table, seq_lens, new_lens, free_pages, free_count, slot_map, positions, cu_new,
                            seq_lens_out, free_left, device_status, D->num_seqs, D->table_width, D->page_size, shift,
                            D->num_free, D->max_new_tokens, D->prefix_len, rows};
    const unsigned grid = (unsigned)std::max<int64_t>(1, (M + rows - 1) / rows);
    if (threads == 256) gdn_kv_extend_kernel<256><<<grid, 256, 0, st>>>(P);
    else gdn_kv_extend_kernel<1024><<<grid, 1024, 0, st>>>(P);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
