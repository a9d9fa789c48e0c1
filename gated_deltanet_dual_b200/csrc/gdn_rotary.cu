// gdn_rotary.cu -- rotary positions (include/gdn_rotary.h) and rotary fused with the append to the
// paged key/value cache (gdn_rotary_append of include/gdn_kvcache.h).
//
// y1 = a (x1 cos t - x2 sin t), y2 = a (x1 sin t + x2 cos t) with t = position * f_i.  The table holds
// f_i / (2 pi) as a 64-bit fraction of a turn, so position * table entry modulo 2^64 is the angle
// with whole turns dropped exactly; its upper 32 bits, as a signed number of half-turns in [-1, 1), go
// to sincospif.  No 64-bit floating point and no slow range reduction on the device.
//
// Bound by memory: every element is read and written once.  A CTA takes a few rows; its threads
// first compute the rows' (cos, sin) once for all heads into shared memory, then each thread keeps
// one column unit (two 16-byte vectors whose elements pair up, or one vector of interleaved
// pairs) and walks over (row, head), a few heads at a time, holding its unit's cos and sin in registers
// within a row.  8 x 4096 rows of 16 + 16 heads of 128 in bf16 take 88.6 us (6.06 TB/s; one read and write at the
// copy rate of 6.46 takes 83.2), gradients of two fp32 views with half of each head in pairs 84 us (78.0), the
// append of 8192 rows 36.0 us (30.9).  More heads at a time cost registers and so CTAs (four in the half
// layout: 126 us).
#include <algorithm>
#include <cmath>

#include "gdn_internal.cuh"
#include "../../include/gdn_kvcache.h"

namespace gdn {
namespace {

constexpr int kRThreads = 256;
constexpr int kRMaxRot = 256;
constexpr int kRMaxRows = 8;         // rows per CTA

struct RotaryParams {
    const void *q, *k, *v;
    void *qo, *ko, *vo;              // append: ko, vo are the caches
    const uint64_t *turns;
    const int32_t *pos, *slots;
    int32_t *status;
    int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, qo_rs, qo_hs, ko_rs, ko_hs;
    int64_t num_slots;
    int32_t rows, npos, H, Hkv, d, rot, rows_per_cta;
    float scale, sign;
};

// The bits of a unit: 16 bytes, or one element; its values as floats, and back with one rounding.
template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}
template <typename T> struct Codec;
template <> struct Codec<float> {
    static __device__ __forceinline__ void get(uint4 u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ void get(uint32_t u, float (&x)[1]) { x[0] = __uint_as_float(u); }
    static __device__ __forceinline__ uint32_t put(const float (&x)[1]) { return __float_as_uint(x[0]); }
};
template <> struct Codec<__nv_bfloat16> {
    static __device__ __forceinline__ void get(uint4 u, float (&x)[8]) {
        x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
        x[4] = bf16_lo(u.z), x[5] = bf16_hi(u.z), x[6] = bf16_lo(u.w), x[7] = bf16_hi(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        return make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
    }
    static __device__ __forceinline__ void get(uint16_t u, float (&x)[1]) { x[0] = bf16_lo(u); }
    static __device__ __forceinline__ uint16_t put(const float (&x)[1]) { return (uint16_t)bf16_pair(x[0], 0.f); }
};
template <typename T, typename R, int N> __device__ __forceinline__ void unpack(R u, float (&x)[N]) { Codec<T>::get(u, x); }
template <typename T, int N> __device__ __forceinline__ auto pack(const float (&x)[N]) { return Codec<T>::put(x); }

// (cos, sin) of one (position, pair), scaled; sin signed.
__device__ __forceinline__ float2 unit_of(int32_t position, uint64_t turn, float scale, float sign) {
    const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(position)) * turn;
    const float half_turns = static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * scale, s * scale * sign);
}

// The head `head` of a row: its source and destination.  Heads [0, H) are q's, [H, H + Hkv) k's and,
// when appending, [H + Hkv, H + 2 Hkv) v's, which are not rotated.
template <typename T, bool APPEND>
struct HeadRef {
    const T *src;
    T *dst;
    bool turn;
    __device__ __forceinline__ HeadRef(const RotaryParams &P, int64_t row, int head, int64_t slot) {
        if (head < P.H) {
            src = static_cast<const T *>(P.q) + row * P.q_rs + head * P.q_hs;
            dst = static_cast<T *>(P.qo) + row * P.qo_rs + head * P.qo_hs;
            turn = true;
        } else if (!APPEND || head < P.H + P.Hkv) {
            const int h = head - P.H;
            src = static_cast<const T *>(P.k) + row * P.k_rs + h * P.k_hs;
            dst = static_cast<T *>(P.ko) + (APPEND ? slot : row) * P.ko_rs + h * P.ko_hs;
            turn = true;
        } else {
            const int h = head - P.H - P.Hkv;
            src = static_cast<const T *>(P.v) + row * P.v_rs + h * P.v_hs;
            dst = static_cast<T *>(P.vo) + slot * P.ko_rs + h * P.ko_hs;
            turn = false;
        }
    }
};

// VEC: units of 16-byte vectors (half layout: two vectors rot/2 apart; interleaved: one vector; the
// part that is not rotated: one vector).  Otherwise units of one pair, or one element of the
// part that is not rotated.
template <typename T, bool IL, bool APPEND, bool VEC>
__global__ void __launch_bounds__(kRThreads) gdn_rotary_kernel(const __grid_constant__ RotaryParams P) {
    __shared__ float2 cs[kRMaxRows * (kRMaxRot / 2)];
    __shared__ int64_t s_slot[kRMaxRows];
    constexpr int VN = VEC ? 16 / (int)sizeof(T) : 1;
    constexpr int PU = !VEC ? 1 : IL ? VN / 2 : VN;         // pairs of a rotated unit
    const int tid = threadIdx.x, np = P.rot >> 1;
    const int64_t row0 = (int64_t)blockIdx.x * P.rows_per_cta;
    const int nrows = (int)min((int64_t)P.rows_per_cta, P.rows - row0);

    if (APPEND && tid < nrows) {
        int64_t slot = P.slots[row0 + tid];
        if (slot < -1 || slot >= P.num_slots) {
            if (P.status) atomicExch(P.status, (int32_t)GDN_ERR_INVALID_ARG);
            slot = -1;
        }
        s_slot[tid] = slot;
    }
    for (int i = tid; i < nrows * np; i += kRThreads) {
        const int r = i / np, pair = i - r * np;
        cs[i] = unit_of(P.pos[(row0 + r) % P.npos], P.turns[pair], P.scale, P.sign);
    }
    __syncthreads();

    const int heads = P.H + P.Hkv * (APPEND ? 2 : 1);
    const int turned = np / PU;                             // rotated units of a head
    const int units = turned + (P.d - P.rot) / VN;
    const int groups = kRThreads / units;
    const int u = tid % units;
    int head = tid / units;
    if (head >= groups) return;
    int row = 0;
    while (head >= heads) {
        head -= heads;
        ++row;
    }
    const bool plain = u >= turned;
    const int e0 = plain ? P.rot + (u - turned) * VN : IL ? u * 2 * PU : u * PU;     // first element
    const int e1 = (IL && !VEC) ? e0 + 1 : e0 + np;         // its partner's (half layout, or scalar pairs)
    float2 w[PU];
    int wrow = -1;
    // kBatch heads at a time: all their loads are on their way before the first store
    constexpr int kBatch = VEC ? (IL ? 4 : 2) : 1;
    constexpr int kBytes = VEC ? 16 : sizeof(T);
    using Raw = typename RawOf<kBytes>::type;
    while (row < nrows) {
        Raw a[kBatch], b[kBatch];
        T *dst[kBatch];
        int rows[kBatch];
        bool turn[kBatch];
        const bool second = !plain && !(IL && VEC);        // the unit's partner lies elsewhere
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            dst[i] = nullptr;
            rows[i] = row;
            turn[i] = false;
            if (row < nrows) {
                const int64_t slot = APPEND ? s_slot[row] : 0;
                if (!APPEND || slot >= 0) {
                    const HeadRef<T, APPEND> h(P, row0 + row, head, slot);
                    dst[i] = h.dst;
                    turn[i] = h.turn && !plain;
                    a[i] = *reinterpret_cast<const Raw *>(h.src + e0);
                    if (second) b[i] = *reinterpret_cast<const Raw *>(h.src + e1);
                }
                head += groups;
                while (head >= heads) {
                    head -= heads;
                    ++row;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (!dst[i]) continue;
            if (turn[i]) {
                if (wrow != rows[i]) {
                    wrow = rows[i];
#pragma unroll
                    for (int j = 0; j < PU; ++j) w[j] = cs[wrow * np + u * PU + j];
                }
                if constexpr (IL && VEC) {
                    float x[VN];
                    unpack<T>(a[i], x);
#pragma unroll
                    for (int j = 0; j < PU; ++j) {
                        const float p = x[2 * j], q = x[2 * j + 1];
                        x[2 * j] = p * w[j].x - q * w[j].y;
                        x[2 * j + 1] = p * w[j].y + q * w[j].x;
                    }
                    a[i] = pack<T>(x);
                } else {
                    float x[VN], y[VN];
                    unpack<T>(a[i], x);
                    unpack<T>(b[i], y);
#pragma unroll
                    for (int j = 0; j < VN; ++j) {
                        const float p = x[j], q = y[j];
                        x[j] = p * w[j].x - q * w[j].y;
                        y[j] = p * w[j].y + q * w[j].x;
                    }
                    a[i] = pack<T>(x);
                    b[i] = pack<T>(y);
                }
            }
            *reinterpret_cast<Raw *>(dst[i] + e0) = a[i];
            if (second) *reinterpret_cast<Raw *>(dst[i] + e1) = b[i];
        }
    }
}

template <typename T, bool IL, bool APPEND>
cudaError_t launch_rotary(const RotaryParams &P, bool vec, cudaStream_t st) {
    const unsigned grid = (unsigned)((P.rows + (int64_t)P.rows_per_cta - 1) / P.rows_per_cta);
    if (vec) gdn_rotary_kernel<T, IL, APPEND, true><<<grid, kRThreads, 0, st>>>(P);
    else gdn_rotary_kernel<T, IL, APPEND, false><<<grid, kRThreads, 0, st>>>(P);
    return cudaGetLastError();
}

template <bool APPEND>
gdn_status run_rotary(RotaryParams &P, int dtype, int interleaved, bool vec, cudaStream_t st) {
    // Rows per CTA: one up to 16 CTAs a SM (a decode step wants every SM), else as many as keep to that number, four
    // waves, so that they share a CTA's set-up; never more than kRMaxRows, for which shared memory has room, so
    // above 18944 rows the CTAs grow in number again (32768 rows: 28 a SM).  Append of 8192 rows: 3 rows (4.6 waves) 37.9 us, 4 rows 36.0, 1 row 45.8.
    P.rows_per_cta = (int)std::min<int64_t>(kRMaxRows, (P.rows + INT64_C(148) * 16 - 1) / (148 * 16));
    cudaError_t e;
    if (dtype == GDN_BF16)
        e = interleaved ? launch_rotary<__nv_bfloat16, true, APPEND>(P, vec, st)
                        : launch_rotary<__nv_bfloat16, false, APPEND>(P, vec, st);
    else
        e = interleaved ? launch_rotary<float, true, APPEND>(P, vec, st) : launch_rotary<float, false, APPEND>(P, vec, st);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

bool multiple(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides of one tensor [rows, heads, d]: non-negative, spanning less than 2^46 elements; an output's
// rows and heads must also lie apart (each stride clears the extent of what is inside it, in either order).
bool strides_ok(int64_t rs, int64_t hs, int64_t rows, int64_t heads, int64_t d, bool output) {
    constexpr int64_t kMost = INT64_C(1) << 46;
    if (rs < 0 || hs < 0) return false;
    if (rows == 0 || heads == 0) return true;
    if ((rows > 1 && rs > kMost / (rows - 1)) || (heads > 1 && hs > kMost / (heads - 1))) return false;
    if (!output) return true;
    const bool heads_inside = (heads <= 1 || hs >= d) && (rows <= 1 || rs >= (heads - 1) * hs + d);
    const bool rows_inside = (rows <= 1 || rs >= d) && (heads <= 1 || hs >= (rows - 1) * rs + d);
    return heads_inside || rows_inside;
}

// The bytes of a tensor [rows, heads, d] (its strides have passed strides_ok).
struct Cover {
    uintptr_t lo;
    int64_t rs, hs, row, all;                   // strides; bytes from a row's first element to its last, and of all rows
    Cover(const void *p, int64_t rows, int64_t rs_, int64_t heads, int64_t hs_, int64_t d, int64_t e)
        : lo(reinterpret_cast<uintptr_t>(p)), rs(rs_ * e), hs(hs_ * e), row(heads ? ((heads - 1) * hs_ + d) * e : 0),
          all(p && rows && heads ? (rows - 1) * rs_ * e + row : 0) {}
    Cover(const void *p, int64_t n, int64_t e) : Cover(p, 1, 0, 1, 0, n, e) {}
    // No byte in common: one lies behind the other, or both have the same row stride and their rows alternate (slices
    // of one projection's output).
    bool apart(const Cover &o) const {
        if (all == 0 || o.all == 0 || lo + all <= o.lo || o.lo + o.all <= lo) return true;
        if (rs != o.rs || rs == 0 || row > rs || o.row > rs) return false;
        const int64_t m = (int64_t)(o.lo - lo) % rs, shift = m < 0 ? m + rs : m;
        return row <= shift && shift + o.row <= rs;
    }
    bool same(const Cover &o) const { return lo == o.lo && rs == o.rs && hs == o.hs; }
};

bool common_ok(int32_t rows, int32_t d, int32_t rot, int32_t il, int32_t dtype, float scale) {
    return rows >= 0 && d >= 1 && rot >= 0 && rot % 2 == 0 && rot <= d && (il == 0 || il == 1) &&
           (dtype == GDN_BF16 || dtype == GDN_FP32) && std::isfinite(scale);
}

// Whether every vector of the fast path is 16-byte aligned and no unit is cut.
struct VecRule {
    int64_t n;          // elements of 16 bytes
    bool ok;
    VecRule(int dtype, int d, int rot, int il) : n(dtype == GDN_BF16 ? 8 : 4) {
        ok = d % n == 0 && rot % (il ? n : 2 * n) == 0;
    }
    void tensor(const void *p, int64_t rs, int64_t hs) {
        if (p) ok = ok && multiple(p, 16) && rs % n == 0 && hs % n == 0;
    }
};

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor,
                                             double original_len, double beta_fast, double beta_slow,
                                             uint64_t *turns_host) {
    if (rot_dim < 0 || rot_dim % 2 || !(base > 0.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) ||
        scaling < GDN_ROPE_NONE || scaling > GDN_ROPE_RAMP)
        return GDN_ERR_INVALID_ARG;
    if (rot_dim > kRMaxRot) return GDN_ERR_UNSUPPORTED;
    if (rot_dim > 0 && !turns_host) return GDN_ERR_INVALID_ARG;
    if (scaling == GDN_ROPE_RAMP && (!(original_len > 0.0) || !std::isfinite(original_len) || !(beta_slow >= 0.0) ||
                                     !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
        return GDN_ERR_INVALID_ARG;
    if (scaling == GDN_ROPE_NTK && rot_dim > 0 && rot_dim < 4) return GDN_ERR_INVALID_ARG;
    const long double two_pi = 6.283185307179586476925286766559005768L;
    long double b = base;
    if (scaling == GDN_ROPE_NTK && rot_dim > 0) b *= powl((long double)factor, (long double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        long double f = powl(b, -2.0L * i / rot_dim);
        if (scaling == GDN_ROPE_LINEAR) f /= factor;
        if (scaling == GDN_ROPE_RAMP) {
            const long double r = original_len * f / two_pi;
            const long double w = std::min(1.0L, std::max(0.0L, (r - beta_slow) / ((long double)beta_fast - beta_slow)));
            f *= w + (1.0L - w) / factor;
        }
        long double turn = f / two_pi;
        if (!std::isfinite(turn)) return GDN_ERR_INVALID_ARG;
        turn -= floorl(turn);
        const long double fixed = roundl(turn * 18446744073709551616.0L);       // 2^64
        turns_host[i] = fixed >= 18446744073709551616.0L ? 0 : (uint64_t)fixed;  // a full turn is none
    }
    return GDN_OK;
}

static gdn_status rotary(const gdn_rotary_desc *D, const uint64_t *turns, const int32_t *positions, const void *q,
                         const void *k, void *q_out, void *k_out, float sign, gdn_stream_t stream) {
    if (!D || !common_ok(D->num_rows, D->head_dim, D->rot_dim, D->interleaved, D->dtype, D->scale) ||
        D->num_positions < 1 || D->num_rows % D->num_positions || D->num_heads < 0 || D->num_kv_heads < 0 ||
        D->num_heads + (int64_t)D->num_kv_heads < 1 || D->num_heads + (int64_t)D->num_kv_heads > INT32_MAX / 2 ||
        D->reserved != 0)
        return GDN_ERR_INVALID_ARG;
    const int64_t R = D->num_rows, d = D->head_dim;
    if (!strides_ok(D->q_row_stride, D->q_head_stride, R, D->num_heads, d, false) ||
        !strides_ok(D->k_row_stride, D->k_head_stride, R, D->num_kv_heads, d, false) ||
        !strides_ok(D->q_out_row_stride, D->q_out_head_stride, R, D->num_heads, d, true) ||
        !strides_ok(D->k_out_row_stride, D->k_out_head_stride, R, D->num_kv_heads, d, true))
        return GDN_ERR_INVALID_ARG;
    if (R == 0) return GDN_OK;
    if ((D->num_heads > 0 && (!q || !q_out)) || (D->num_kv_heads > 0 && (!k || !k_out)) ||
        (D->rot_dim > 0 && (!turns || !positions)))
        return GDN_ERR_INVALID_ARG;
    const bool in_place_ok =
        (q != q_out || !q || (D->q_row_stride == D->q_out_row_stride && D->q_head_stride == D->q_out_head_stride)) &&
        (k != k_out || !k || (D->k_row_stride == D->k_out_row_stride && D->k_head_stride == D->k_out_head_stride));
    if (!in_place_ok) return GDN_ERR_INVALID_ARG;
    const uintptr_t e = D->dtype == GDN_BF16 ? 2 : 4;
    if (!multiple(positions, 4) || !multiple(turns, 8) || !multiple(q, e) || !multiple(k, e) || !multiple(q_out, e) ||
        !multiple(k_out, e))
        return GDN_ERR_ALIGNMENT;
    if (D->head_dim > kRMaxRot) return GDN_ERR_UNSUPPORTED;
    const int64_t H = D->num_heads, Hkv = D->num_kv_heads, es = e;
    const Cover cq(q, R, D->q_row_stride, H, D->q_head_stride, d, es), ck(k, R, D->k_row_stride, Hkv, D->k_head_stride, d, es),
        cqo(q_out, R, D->q_out_row_stride, H, D->q_out_head_stride, d, es),
        cko(k_out, R, D->k_out_row_stride, Hkv, D->k_out_head_stride, d, es), cpos(positions, D->num_positions, 4),
        cturns(turns, D->rot_dim / 2, 8);
    if (!(cqo.same(cq) || cqo.apart(cq)) || !(cko.same(ck) || cko.apart(ck)) || !cqo.apart(ck) || !cko.apart(cq) ||
        !cqo.apart(cko) || !cqo.apart(cpos) || !cko.apart(cpos) || !cqo.apart(cturns) || !cko.apart(cturns))
        return GDN_ERR_INVALID_ARG;
    RotaryParams P = {};
    P.q = q, P.k = k, P.qo = q_out, P.ko = k_out;
    P.turns = turns, P.pos = positions;
    P.q_rs = D->q_row_stride, P.q_hs = D->q_head_stride, P.k_rs = D->k_row_stride, P.k_hs = D->k_head_stride;
    P.qo_rs = D->q_out_row_stride, P.qo_hs = D->q_out_head_stride;
    P.ko_rs = D->k_out_row_stride, P.ko_hs = D->k_out_head_stride;
    P.rows = D->num_rows, P.npos = D->num_positions, P.H = D->num_heads, P.Hkv = D->num_kv_heads;
    P.d = D->head_dim, P.rot = D->rot_dim, P.scale = D->scale, P.sign = sign;
    VecRule rule(D->dtype, P.d, P.rot, D->interleaved);
    if (P.H) rule.tensor(q, P.q_rs, P.q_hs), rule.tensor(q_out, P.qo_rs, P.qo_hs);
    if (P.Hkv) rule.tensor(k, P.k_rs, P.k_hs), rule.tensor(k_out, P.ko_rs, P.ko_hs);
    return run_rotary<false>(P, D->dtype, D->interleaved, rule.ok, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" gdn_status gdn_rotary_forward(const gdn_rotary_desc *desc, const uint64_t *turns, const int32_t *positions,
                                         const void *q, const void *k, void *q_out, void *k_out, gdn_stream_t stream) {
    return rotary(desc, turns, positions, q, k, q_out, k_out, 1.f, stream);
}

extern "C" gdn_status gdn_rotary_backward(const gdn_rotary_desc *desc, const uint64_t *turns, const int32_t *positions,
                                          const void *q, const void *k, void *q_out, void *k_out, gdn_stream_t stream) {
    return rotary(desc, turns, positions, q, k, q_out, k_out, -1.f, stream);
}

extern "C" gdn_status gdn_rotary_append(const gdn_append_desc *D, const uint64_t *turns, const int32_t *positions,
                                        const int32_t *slot_map, const void *q, const void *k, const void *v,
                                        void *q_out, void *k_cache, void *v_cache, int32_t *device_status,
                                        gdn_stream_t stream) {
    if (!D || !common_ok(D->num_rows, D->head_dim, D->rot_dim, D->interleaved, D->dtype, D->scale) || D->num_heads < 1 ||
        D->num_kv_heads < 1 || D->num_heads + 2 * (int64_t)D->num_kv_heads > INT32_MAX / 2 || D->page_size < 1 ||
        D->num_pages < 1 || (int64_t)D->page_size * D->num_pages > INT32_MAX)
        return GDN_ERR_INVALID_ARG;
    const int64_t R = D->num_rows, d = D->head_dim;
    if (!strides_ok(D->q_row_stride, D->q_head_stride, R, D->num_heads, d, false) ||
        !strides_ok(D->k_row_stride, D->k_head_stride, R, D->num_kv_heads, d, false) ||
        !strides_ok(D->v_row_stride, D->v_head_stride, R, D->num_kv_heads, d, false) ||
        !strides_ok(D->q_out_row_stride, D->q_out_head_stride, R, D->num_heads, d, true))
        return GDN_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || (R > 0 && (!slot_map || !q || !k || !v || !q_out || (D->rot_dim > 0 && (!turns || !positions)))))
        return GDN_ERR_INVALID_ARG;
    if (R > 0 && q == q_out && (D->q_row_stride != D->q_out_row_stride || D->q_head_stride != D->q_out_head_stride))
        return GDN_ERR_INVALID_ARG;
    const uintptr_t e = D->dtype == GDN_BF16 ? 2 : 4;
    if (!multiple(positions, 4) || !multiple(slot_map, 4) || !multiple(turns, 8) || !multiple(q, e) || !multiple(k, e) ||
        !multiple(v, e) || !multiple(q_out, e) || !multiple(k_cache, e) || !multiple(v_cache, e) || !multiple(device_status, 4))
        return GDN_ERR_ALIGNMENT;
    if (D->head_dim > kRMaxRot) return GDN_ERR_UNSUPPORTED;
    const int64_t Hkv = D->num_kv_heads, es = e, slots = (int64_t)D->page_size * D->num_pages;
    const Cover cq(q, R, D->q_row_stride, D->num_heads, D->q_head_stride, d, es),
        cqo(q_out, R, D->q_out_row_stride, D->num_heads, D->q_out_head_stride, d, es),
        in[] = {{k, R, D->k_row_stride, Hkv, D->k_head_stride, d, es}, {v, R, D->v_row_stride, Hkv, D->v_head_stride, d, es},
                {positions, R, 4}, {slot_map, R, 4}, {turns, D->rot_dim / 2, 8}},
        out[] = {cqo, {k_cache, slots, Hkv * d, Hkv, d, d, es}, {v_cache, slots, Hkv * d, Hkv, d, d, es}, {device_status, 1, 4}};
    if (!cqo.same(cq) && !cqo.apart(cq)) return GDN_ERR_INVALID_ARG;
    for (const Cover &o : out) {
        if (&o != out && !o.apart(cq)) return GDN_ERR_INVALID_ARG;
        for (const Cover &i : in)
            if (!o.apart(i)) return GDN_ERR_INVALID_ARG;
        for (const Cover &x : out)
            if (&x != &o && !o.apart(x)) return GDN_ERR_INVALID_ARG;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (device_status && cudaMemsetAsync(device_status, 0, sizeof(int32_t), st) != cudaSuccess) return GDN_ERR_CUDA;
    if (R == 0) return GDN_OK;
    RotaryParams P = {};
    P.q = q, P.k = k, P.v = v, P.qo = q_out, P.ko = k_cache, P.vo = v_cache;
    P.turns = turns, P.pos = positions, P.slots = slot_map, P.status = device_status;
    P.q_rs = D->q_row_stride, P.q_hs = D->q_head_stride, P.k_rs = D->k_row_stride, P.k_hs = D->k_head_stride;
    P.v_rs = D->v_row_stride, P.v_hs = D->v_head_stride;
    P.qo_rs = D->q_out_row_stride, P.qo_hs = D->q_out_head_stride;
    P.ko_rs = (int64_t)D->num_kv_heads * d, P.ko_hs = d;
    P.num_slots = (int64_t)D->page_size * D->num_pages;
    P.rows = D->num_rows, P.npos = D->num_rows, P.H = D->num_heads, P.Hkv = D->num_kv_heads;
    P.d = D->head_dim, P.rot = D->rot_dim, P.scale = D->scale, P.sign = 1.f;
    VecRule rule(D->dtype, P.d, P.rot, D->interleaved);
    rule.tensor(q, P.q_rs, P.q_hs), rule.tensor(q_out, P.qo_rs, P.qo_hs), rule.tensor(k, P.k_rs, P.k_hs);
    rule.tensor(v, P.v_rs, P.v_hs), rule.tensor(k_cache, P.ko_rs, P.ko_hs), rule.tensor(v_cache, P.ko_rs, P.ko_hs);
    return run_rotary<true>(P, D->dtype, D->interleaved, rule.ok, st);
}
