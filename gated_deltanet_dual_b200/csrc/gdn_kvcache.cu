// gdn_kvcache.cu -- block tables, slots and positions of a serving step's new tokens
// (gdn_kv_extend of include/gdn_kvcache.h).
//
// Two exclusive sums over the sequences -- pages needed and tokens -- decide everything: which
// entry of the free list a new page takes and which packed row a token has.  A few kilobytes are
// read and 8 bytes per token written, so the call is bound by latency: one launch, in which every
// CTA runs the whole scan itself (4096 sequences per pass of 1024 threads; the lengths come from
// L2) and then writes only its own range of token rows.  A token whose index starts a page also
// writes that page's table entry, so entries have one writer and no CTA reads an entry that
// another one writes (rows on new pages take the page from the free list).
#include <algorithm>
#include <climits>

#include "gdn_internal.cuh"
#include "../../include/gdn_kvcache.h"

namespace gdn {
namespace {

constexpr int kXThreads = 1024;
constexpr int kXItems = 4;                      // sequences per thread and pass
constexpr int kXPass = kXThreads * kXItems;
constexpr int kXRows = 4096;                    // most token rows of a CTA
constexpr int kXDirect = 4;                     // a thread writes so many of its sequence's rows by itself
constexpr int kXList = kXRows / (kXDirect + 1) + 2;

struct ExtendParams {
    int32_t *table;
    const int32_t *lens, *fresh, *free_pages, *free_count;
    int32_t *slot_map, *positions, *cu, *lens_out, *free_left, *status;
    int32_t N, W, page, F, M, prefix, rows_per_cta;
};

// One sequence's rows: n < 0 marks a refused one.
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
    const int j = i / P.page, off = i - j * P.page;
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

__global__ void __launch_bounds__(kXThreads) gdn_kv_extend_kernel(const ExtendParams P) {
    __shared__ int64_t s_need[32], s_new[32];
    __shared__ Run s_list[kXList];
    __shared__ int s_count;
    __shared__ unsigned long long s_taken;      // pages that served sequences take
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row0 = (int)min((int64_t)blockIdx.x * P.rows_per_cta, (int64_t)P.M);
    const int row1 = (int)min((int64_t)row0 + P.rows_per_cta, (int64_t)P.M);
    const int32_t count = *P.free_count;
    const int top = min(max(count, 0), P.F);
    bool bad = top != count;
    int64_t need_before = 0, new_before = 0;    // sums of the earlier passes
    if (tid == 0) s_taken = 0;

    for (int base = 0, pass = 0; base < P.N; base += kXPass, ++pass) {
        int32_t len[kXItems], w[kXItems], have[kXItems], need[kXItems];
        bool wrong[kXItems];
        int64_t my_need = 0, my_new = 0;
        const int n0 = base + tid * kXItems;
#pragma unroll
        for (int i = 0; i < kXItems; ++i) {
            const bool in = n0 + i < P.N;
            len[i] = in ? P.lens[n0 + i] : 0;
            w[i] = in ? P.fresh[n0 + i] : 0;
        }
#pragma unroll
        for (int i = 0; i < kXItems; ++i) {
            wrong[i] = len[i] < 0 || w[i] < 0 || (int64_t)len[i] + w[i] > (int64_t)P.W * P.page;
            w[i] = max(w[i], 0);
            my_new += w[i];
        }
        // tokens first: a sequence whose rows pass M takes no pages
        int64_t x = my_new;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();                        // the last pass has read s_new, s_need and the list
        if (tid == 0) s_count = 0;
        if (lane == 31) s_new[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int64_t t = s_new[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += y;
            }
            s_new[lane] = t;
        }
        __syncthreads();
        int64_t cu = new_before + x - my_new + (warp ? s_new[warp - 1] : 0);
        new_before += s_new[31];
        {
            int64_t c = cu;
#pragma unroll
            for (int i = 0; i < kXItems; ++i) {
                c += w[i];
                wrong[i] = wrong[i] || c > P.M;
                have[i] = wrong[i] ? 0 : (int)(((int64_t)len[i] + P.page - 1) / P.page);
                need[i] = wrong[i] ? 0 : (int)(((int64_t)len[i] + w[i] + P.page - 1) / P.page) - have[i];
                my_need += need[i];
            }
        }
        x = my_need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_need[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int64_t t = s_need[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += y;
            }
            s_need[lane] = t;
        }
        __syncthreads();
        int64_t before = need_before + x - my_need + (warp ? s_need[warp - 1] : 0);
        need_before += s_need[31];

        const bool writer = pass % gridDim.x == blockIdx.x;     // this pass's per-sequence outputs
#pragma unroll
        for (int i = 0; i < kXItems; ++i) {
            const int n = n0 + i;
            if (n < P.N) {
                Run r;
                r.cu = cu, r.page0 = before, r.n = n, r.len = len[i], r.have = have[i];
                r.refused = wrong[i] || (need[i] > 0 && before + need[i] > top);
                r.lo = (int)min(max(cu, (int64_t)row0), (int64_t)row1);
                r.hi = (int)min(cu + w[i], (int64_t)row1);
                if (r.refused) bad = true;
                else if (need[i] > 0) atomicMax(&s_taken, (unsigned long long)(before + need[i]));
                if (writer) {
                    P.cu[n] = (int32_t)min(cu, (int64_t)INT32_MAX);
                    P.lens_out[n] = r.refused ? len[i] : len[i] + w[i];
                }
                if (r.hi - r.lo > kXDirect) s_list[atomicAdd(&s_count, 1)] = r;
                else
                    for (int row = r.lo; row < r.hi; ++row) write_row(P, r, row, top);
                cu += w[i];
                before += need[i];
            }
        }
        __syncthreads();
        const int listed = s_count;
        for (int e = warp; e < listed; e += kXThreads / 32) {               // short runs: a warp each
            const Run r = s_list[e];
            if (r.hi - r.lo <= 256)
                for (int row = r.lo + lane; row < r.hi; row += 32) write_row(P, r, row, top);
        }
        for (int e = 0; e < listed; ++e) {                                  // long ones: the CTA
            if (s_list[e].hi - s_list[e].lo <= 256) continue;
            const Run r = s_list[e];
            for (int row = r.lo + tid; row < r.hi; row += kXThreads) write_row(P, r, row, top);
        }
    }
    for (int64_t row = max(new_before, (int64_t)row0) + tid; row < row1; row += kXThreads) {     // padding rows
        P.slot_map[row] = -1;
        P.positions[row] = -1;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (tid == 0) {
            P.cu[P.N] = (int32_t)min(new_before, (int64_t)INT32_MAX);
            *P.free_left = top - (int)s_taken;
        }
        if (bad && P.status) atomicExch(P.status, (int32_t)GDN_ERR_INVALID_ARG);
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
        D->prefix_len < 0 || D->reserved[0] || D->reserved[1] || D->num_seqs > INT32_MAX - 2 * kXPass)
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
    ExtendParams P = {block_table, seq_lens, new_lens, free_pages, free_count, slot_map, positions, cu_new, seq_lens_out,
                      free_left, device_status, D->num_seqs, D->table_width, D->page_size, D->num_free,
                      D->max_new_tokens, D->prefix_len, 0};
    // token rows per CTA: a CTA's threads' worth, more only when that would pass one CTA per SM
    P.rows_per_cta = (int)std::min<int64_t>(kXRows, std::max<int64_t>(kXThreads, (M + 147) / 148));
    const unsigned grid = (unsigned)std::max<int64_t>(1, (M + P.rows_per_cta - 1) / P.rows_per_cta);
    gdn_kv_extend_kernel<<<grid, kXThreads, 0, st>>>(P);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
