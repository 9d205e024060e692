// experts.hip -- MXFP4 rows, the grouped MXFP4 product of the local experts
// and the MoE layer of a few tokens, for MI355X (gfx950).  Included after
// cdl.hip (same translation unit).
//
// MXFP4 (OCP microscaling): groups of 32 elements along a row share a scale
// 2^e, stored as the byte e + 127; an element is an e2m1 code (sign, 2
// exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte,
// the even element in the low half.

#include <type_traits>

namespace {

// ---------------------------------------------------------------------------
// MXFP4 quantisation
// ---------------------------------------------------------------------------

typedef __bf16 v2bf16 __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Two fp32 values to a pair of bf16, round to nearest even: one
// v_cvt_pk_bf16_f32 (any NaN stays one; the dispatch's own conversion also
// fixes its pattern, at several instructions a value).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, v2bf16{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// The scale byte of a group from the bits of its largest magnitude as a
// bf16 (16 bits): the smallest power of two 2^(b - 127), b >= 0, with
// 6 * 2^(b - 127) >= amax.  amax = 1.f * 2^(E - 127) and 6 = 1.5 * 2^2, so
// b = E - 2 when 1.f <= 1.5 and E - 1 otherwise (subnormals and the smallest
// normals give 0: 6 * 2^-127 covers them).  An infinite amax takes 254, the
// largest scale: 6 * 2^127 reads back as infinity.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax16)
{
    const int E = (int)(amax16 >> 7);
    if (E == 255) return 254u;
    const int b = E - 2 + ((amax16 & 0x7Fu) > 0x40u ? 1 : 0);
    return (uint32_t)(b < 0 ? 0 : b);
}

// 16 consecutive bf16 of a row (two 16-byte chunks) to 16 codes (8 bytes);
// the 2 lanes of an even-odd pair hold one group.  *scale receives the
// group's byte in both lanes.  A group with a NaN takes the scale's NaN code
// (255) and zero codes, so that the whole group reads back as NaN.
// v_cvt_scalef32_pk_fp4_bf16 rounds x / 2^E to the nearest code, ties to the
// even one, with E the exponent field of its scale operand read as an E8M0
// code (field 0: 2^-127), and saturates at 6; checked on gfx950 for eleven
// fields from 0 to 254 over every bf16 of up to 2^56 times the scale.  The
// byte chosen here leaves no finite magnitude above 6 times the scale.
__device__ __forceinline__ u32x2 mx_quant16(u32x4 a, u32x4 b, uint32_t *scale)
{
    using u16x2 = unsigned short __attribute__((ext_vector_type(2)));
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    u16x2 m = __builtin_bit_cast(u16x2, w[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
    const uint32_t am = dpp_umax_step<0xB1>((uint32_t)(m.x > m.y ? m.x : m.y));   // the pair's other lane
    const bool nan = am > kBf16ExpMask;       // NaN magnitudes order above infinity's
    const uint32_t byte = mx_scale_byte(am);
    const float p = __uint_as_float(byte << 23);
    uint32_t q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf16, w[4 * i]), p, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf16, w[4 * i + 1]), p, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf16, w[4 * i + 2]), p, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2bf16, w[4 * i + 3]), p, 3);
        q[i] = nan ? 0u : r;
    }
    *scale = nan ? 255u : byte;
    return u32x2{q[0], q[1]};
}

__device__ __forceinline__ uint64_t lanes_below(int lane) { return lane ? ~0ull >> (kWave - lane) : 0ull; }

constexpr int kMxPairs = 7;      // blocks of 1024 elements a wave holds: one row at H = 7168

// A wave's row from element `first` on (a multiple of 7 blocks), 7 blocks of
// 1024 elements: lane l has elements 1024 p + 16 l to + 15 of block p, q[p]
// their codes; the even lanes hold their groups' scale bytes in s[p].
struct MxRow {
    u32x2 q[kMxPairs];
    uint32_t s[kMxPairs];

    __device__ __forceinline__ void load_quant(rsrc_t xr, int lane, uint32_t first)
    {
        u32x4 v[2 * kMxPairs];
#pragma unroll
        for (int p = 0; p < kMxPairs; ++p) {
            v[2 * p] = buf_ld16(xr, (uint32_t)lane * 32u + p * 2048u + first * 2u, 0);
            v[2 * p + 1] = buf_ld16(xr, (uint32_t)lane * 32u + p * 2048u + first * 2u + 16u, 0);
        }
#pragma unroll
        for (int p = 0; p < kMxPairs; ++p) q[p] = mx_quant16(v[2 * p], v[2 * p + 1], &s[p]);
    }

    // The scales as words (four bytes of neighbouring groups): lane 8 d + p
    // takes word d of block p, so that all of them leave in one store.
    __device__ __forceinline__ uint32_t scale_words(int lane) const
    {
        uint32_t mine = 0;
#pragma unroll
        for (int p = 0; p < kMxPairs; ++p) {
            const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s[p], 0x00, 0xF, 0xF, false);   // quad_perm [0,0,0,0]
            const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s[p], 0xAA, 0xF, 0xF, false);   // quad_perm [2,2,2,2]
            const uint32_t w = lo | hi << 8;
            const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x141, 0xF, 0xF, false);      // row_half_mirror
            const uint32_t word = lane & 4 ? o | w << 16 : w | o << 16;
            mine = (lane & 7) == p ? word : mine;
        }
        return mine;
    }

    // To row dst.  The range check of the row's descriptors drops the lanes
    // past the row (H is a multiple of 32: a lane's 8 bytes and its group's
    // byte are inside the row or outside as a whole).  words: scale rows are
    // word-aligned, and `sw` is scale_words().
    __device__ __forceinline__ void store(int lane, uint8_t *oq, uint8_t *os, int64_t dst, int64_t H, uint32_t first,
                                          bool words, uint32_t sw) const
    {
        const rsrc_t rq = make_rsrc(oq + dst * (H / 2), (uint32_t)(H / 2));
        const rsrc_t rs = make_rsrc(os + dst * (H / 32), (uint32_t)(H / 32));
#pragma unroll
        for (int p = 0; p < kMxPairs; ++p) {
            if ((int64_t)first + p * 1024 >= H) break;
            __builtin_amdgcn_raw_buffer_store_b64(q[p], rq, (uint32_t)lane * 8u + p * 512u + first / 2, 0, 0);
            if (!words && (lane & 1) == 0)
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)s[p], rs, (uint32_t)lane / 2 + p * 32u + first / 32, 0, 0);
        }
        if (words && (lane & 7) < kMxPairs)
            __builtin_amdgcn_raw_buffer_store_b32(sw, rs, (uint32_t)((lane & 7) * 8 + (lane >> 3)) * 4u + first / 32, 0, 0);
    }
};

__device__ __forceinline__ bool mx_scale_rows_aligned(const uint8_t *os, int64_t H)
{
    return (H / 32) % 4 == 0 && ((uintptr_t)os & 3) == 0;
}

constexpr int kMxRowsPerWg = 4;      // rows (waves) per workgroup

// Rows quantised in place order: out row r from x row r.
__global__ __launch_bounds__(kMxRowsPerWg *kWave) void mx_quant_kernel(
    const uint16_t *__restrict__ x, int64_t rows, int64_t H, uint8_t *__restrict__ q, uint8_t *__restrict__ s)
{
    const int lane = threadIdx.x & (kWave - 1);
    const bool words = mx_scale_rows_aligned(s, H);
    for (int64_t r = (int64_t)blockIdx.x * kMxRowsPerWg + wave_id(); r < rows;
         r += (int64_t)gridDim.x * kMxRowsPerWg) {
        const rsrc_t xr = make_rsrc(x + r * H, (uint32_t)(H * 2));
        for (uint32_t first = 0; (int64_t)first < H; first += kMxPairs * 1024) {
            MxRow row;
            row.load_quant(xr, lane, first);
            row.store(lane, q, s, r, H, first, words, words ? row.scale_words(lane) : 0u);
        }
    }
}

// Codes back to bf16 (exact: three significant bits, exponents in bf16's
// range; 6 * 2^127 and 4 * 2^126 overflow to infinity).  8 elements a thread
// and step, so that a wave stores 1 KB of a row at once.
constexpr int kMxDequantSteps = 4;
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint32_t *__restrict__ q, const uint8_t *__restrict__ s,
                                                         int64_t n8, u32x4 *__restrict__ out)
{
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * kMxDequantSteps) + threadIdx.x; i0 < n8;
         i0 += (int64_t)gridDim.x * (256 * kMxDequantSteps)) {
        uint32_t c[kMxDequantSteps], e[kMxDequantSteps];
#pragma unroll
        for (int j = 0; j < kMxDequantSteps; ++j) {
            const int64_t i = i0 + j * 256;
            c[j] = i < n8 ? q[i] : 0u;
            e[j] = i < n8 ? s[i >> 2] : 0u;
        }
#pragma unroll
        for (int j = 0; j < kMxDequantSteps; ++j) {
            const int64_t i = i0 + j * 256;
            const float p = __uint_as_float(e[j] << 23);
            const u32x4 o = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], p, 0)),
                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], p, 1)),
                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], p, 2)),
                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j], p, 3))};
            if (i < n8) __builtin_nontemporal_store(o, out + i);
        }
    }
}

// Token t's row to the destinations in dmask (lane j holds slot j's): the
// part already held, when there is one, then the others.
__device__ __forceinline__ void mx_store_token(const uint16_t *x, int64_t t, int64_t H, int lane, uint8_t *oq,
                                               uint8_t *os, int32_t d, uint64_t dmask, uint32_t next, const MxRow *held)
{
    if (dmask == 0) return;
    const bool words = mx_scale_rows_aligned(os, H);
    auto store = [&](const MxRow &row, uint32_t first) {
        const uint32_t sw = words ? row.scale_words(lane) : 0u;
        for (uint64_t m = dmask; m; m &= m - 1)
            row.store(lane, oq, os, __builtin_amdgcn_readlane(d, (int)__builtin_ctzll(m)), H, first, words, sw);
    };
    if (held) store(*held, 0);
    const rsrc_t xr = make_rsrc(x + t * H, (uint32_t)(H * 2));
    for (; (int64_t)next < H; next += kMxPairs * 1024) {
        MxRow row;
        row.load_quant(xr, lane, next);
        store(row, next);
    }
}

// Where the scatter puts a row in the padded low-latency buffer.
struct MxLL {
    const int32_t *ids;
    int32_t expert_begin;
    int32_t L;
    const int64_t *seg_indptr;
    const int32_t *counts;
    int64_t cap;
    int32_t *masked_m;
    int32_t *ll_src2dst;
};

// Scatter from a given layout, one wave per token: the row is quantised once
// and stored to every destination (lane j holds slot j's).
template <bool LL>
__global__ __launch_bounds__(kMxRowsPerWg *kWave) void mx_scatter_kernel(
    const uint16_t *__restrict__ x, int64_t T, int64_t H, int32_t k, const int32_t *__restrict__ src2dst,
    uint8_t *__restrict__ oq, uint8_t *__restrict__ os, int64_t cap_rows, int32_t *__restrict__ status, MxLL ll)
{
    const int lane = threadIdx.x & (kWave - 1);
    if constexpr (LL) {
        if (blockIdx.x == 0)
            for (int e = threadIdx.x; e < ll.L; e += kMxRowsPerWg * kWave) {
                const int64_t c = ll.counts[e];
                ll.masked_m[e] = (int32_t)(c < ll.cap ? c : ll.cap);
            }
    }
    const int64_t t = (int64_t)blockIdx.x * kMxRowsPerWg + wave_id();
    if (t >= T) return;
    int32_t d = lane < k ? src2dst[t * k + lane] : -1;
    bool drop = false;
    if constexpr (LL) {
        if (lane < k) {
            const int32_t e = d >= 0 ? local_expert(ll.ids[t * k + lane], ll.expert_begin, ll.L) : -1;
            if (e >= 0) {
                const int64_t slot = d - ll.seg_indptr[e];
                drop = slot >= ll.cap;
                d = drop ? -1 : (int32_t)(e * ll.cap + slot);
            } else {
                d = -1;
            }
            ll.ll_src2dst[t * k + lane] = d;
        }
        if (__ballot(drop) != 0 && lane == 0) set_status(status, CDL_STATUS_LL_OVERFLOW);
    } else {
        drop = d >= 0 && (int64_t)d >= cap_rows;
        if (__ballot(drop) != 0 && lane == 0) set_status(status, CDL_STATUS_ROWS_OVERFLOW);
        if (drop) d = -1;
    }
    mx_store_token(x, t, H, lane, oq, os, d, __ballot(d >= 0), 0, nullptr);
}

// One wave's layout of a small batch without superblock counts: as
// layout_one_wave, with every slot counted here; tot[] is left holding the
// experts' first rows.
template <int TPB>
__device__ __forceinline__ void mx_layout_self(const PermuteArgs &a, int64_t blk, int32_t *tot, int32_t *cur,
                                               int32_t *dsts)
{
    constexpr int kLB = 16;
    const int L = a.L, k = a.k, lane = threadIdx.x & (kWave - 1);
    const int n = (int)(a.T * k);
    const int64_t t_end = (blk + 1) * TPB < a.T ? (blk + 1) * TPB : a.T;
    const int begin = (int)(blk * TPB * k), end = (int)(t_end * k);
    const rsrc_t r_ids = make_rsrc(a.ids, (uint32_t)n * 4u);
    int32_t my[TPB];
#pragma unroll
    for (int r = 0; r < TPB; ++r) my[r] = buf_ld4(r_ids, (uint32_t)(begin + r * kWave + lane) * 4u, 0);
    for (int e = lane; e < L; e += kWave) tot[e] = cur[e] = 0;
    for (int b0 = 0; b0 < n; b0 += kWave * kLB) {
        int32_t id[kLB];
#pragma unroll
        for (int q = 0; q < kLB; ++q) id[q] = buf_ld4(r_ids, (uint32_t)(b0 + q * kWave + lane) * 4u, 0);
#pragma unroll
        for (int q = 0; q < kLB; ++q) {
            const int i = b0 + q * kWave + lane;
            const int32_t e = i < n ? local_expert(id[q], a.expert_begin, L) : -1;
            if (e >= 0) {
                atomicAdd(&tot[e], 1);
                if (i < begin) atomicAdd(&cur[e], 1);
            }
        }
    }
    // the experts' padded offsets; workgroup 0 publishes, the padding rows are shared out
    const int A = a.alignment;
    const int nblk = (int)((a.T + TPB - 1) / TPB);
    int32_t base = 0;
    for (int e0 = 0; e0 < L; e0 += kWave) {
        const int e = e0 + lane;
        const int32_t cnt = e < L ? tot[e] : 0;
        const int32_t padded = (cnt + A - 1) / A * A;
        const int32_t incl = wave_inclusive_scan(padded);
        const int32_t excl = base + incl - padded;
        if (e < L) {
            if (blk == 0) {
                a.counts[e] = cnt;
                a.seg_indptr[e] = excl;
                if (a.masked_m) a.masked_m[e] = (int32_t)(cnt < a.ll_cap ? cnt : a.ll_cap);
            }
            cur[e] += excl;
            tot[e] = excl;
            if (e % nblk == (int)blk)
                for (int64_t r = excl + cnt; r < excl + padded && r < a.reorder_cap; ++r) a.reorder[r] = -1;
        }
        base += __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    if (blk == 0 && lane == 0) {
        a.seg_indptr[L] = base;
        if ((int64_t)base > a.reorder_cap) set_status(a.status, CDL_STATUS_REORDER_OVERFLOW);
    }
    // stable ranks, 64 slots a round
#pragma unroll
    for (int r = 0; r < TPB; ++r) {
        const int i = begin + r * kWave + lane;
        if (begin + r * kWave >= end) break;
        const int32_t e = i < end ? local_expert(my[r], a.expert_begin, L) : -1;
        uint64_t pending = __ballot(e >= 0);
        int32_t dst = -1;
        while (pending) {
            const int leader = __builtin_ctzll(pending);
            const int32_t el = __builtin_amdgcn_readlane(e, leader);
            const uint64_t m = __ballot(e == el);
            const int32_t before = cur[el];
            if (e == el) dst = before + __popcll(m & lanes_below(lane));
            if (lane == leader) cur[el] = before + __popcll(m);
            pending &= ~m;
        }
        if (i < end) {
            a.src2dst[i] = dst;
            if (dst >= 0 && (int64_t)dst < a.reorder_cap) a.reorder[dst] = e;
            dsts[r * kWave + lane] = dst;
        }
    }
}

// Layout and scatter in one launch (two with superblock counts): TPB row waves
// quantise their tokens' rows while one more wave derives the workgroup's
// destinations; after the one barrier the row waves store.  SELF: a small
// batch, whose layout wave counts every slot itself; of up to 512 tokens (one a
// workgroup) the rows are loaded without first looking for a local slot.
template <int TPB, bool SELF, bool LL>
__global__ __launch_bounds__((TPB + 1) * kWave) void mx_permute_kernel(PermuteArgs a, const uint16_t *__restrict__ x,
                                                                      int64_t H, uint8_t *__restrict__ oq,
                                                                      uint8_t *__restrict__ os)
{
    static_assert(SELF || !LL, "the padded form of a large batch scatters from a given layout");
    extern __shared__ int32_t lds[];
    const int L = a.L, k = a.k, lane = threadIdx.x & (kWave - 1), wave = wave_id();
    int32_t *tot = lds, *cur = lds + L, *dsts = lds + 2 * L;
    const int64_t t = (int64_t)blockIdx.x * TPB + wave;
    const bool real = wave < TPB && t < a.T;
    int32_t id = 0;
    bool row = false;
    MxRow held;
    if (wave == TPB) {
        if constexpr (SELF)
            mx_layout_self<TPB>(a, blockIdx.x, tot, cur, dsts);
        else
            layout_one_wave<TPB>(a, blockIdx.x, tot, cur, dsts);
    } else if (real) {
        const rsrc_t r_tok = make_rsrc(a.ids + t * k, (uint32_t)k * 4u);
        id = buf_ld4(r_tok, (uint32_t)lane * 4u, 0);
        row = (SELF && TPB == 1) || __ballot(lane < k && local_expert(id, a.expert_begin, L) >= 0) != 0;
        if (row) held.load_quant(make_rsrc(x + t * H, (uint32_t)(H * 2)), lane, 0);
    }
    __syncthreads();
    if (!(LL ? real : row)) return;            // (a padded form's map names every slot; without a row none is stored)
    int32_t d = lane < k ? dsts[wave * k + lane] : -1;
    bool drop = false;
    if constexpr (LL) {
        const int32_t e = d >= 0 ? local_expert(id, a.expert_begin, L) : 0;
        const int64_t slot = d >= 0 ? d - tot[e] : 0;
        drop = d >= 0 && slot >= a.ll_cap;
        d = d < 0 || drop ? -1 : (int32_t)(e * a.ll_cap + slot);
        if (lane < k) a.ll_src2dst[t * k + lane] = d;
        if (__ballot(drop) != 0 && lane == 0) set_status(a.status, CDL_STATUS_LL_OVERFLOW);
    } else {
        drop = d >= 0 && (int64_t)d >= a.cap_rows;
        if (__ballot(drop) != 0 && lane == 0) set_status(a.status, CDL_STATUS_ROWS_OVERFLOW);
        if (drop) d = -1;
    }
    mx_store_token(x, t, H, lane, oq, os, d, __ballot(d >= 0), kMxPairs * 1024, &held);
}

// ---------------------------------------------------------------------------
// grouped MXFP4 product
// ---------------------------------------------------------------------------

struct GroupedArgs {
    const uint8_t *q;            // [rows, K / 2]
    const uint8_t *s;            // [rows, K / 32]
    int64_t rows;
    int64_t K;
    const uint8_t *wq;           // [L, N, K / 2]
    const uint8_t *ws;           // [L, N, K / 32]
    int32_t L;
    int64_t N;                   // weight rows (2 I for SwiGLU)
    const int32_t *counts;
    const int64_t *seg;          // NULL: expert e's rows start at e * cap
    int64_t cap;
    int32_t *status;
    uint16_t *out;               // [rows, N] bf16
    uint8_t *hq;                 // SwiGLU: [rows, I / 2], [rows, I / 32]
    uint8_t *hs;
};

// Expert e's first row and its row count, held inside the buffer whatever
// the device arrays say.
__device__ __forceinline__ int64_t grouped_rows(const GroupedArgs &a, int e, int64_t *begin, bool *bad)
{
    int64_t c = a.counts[e], b = a.seg ? a.seg[e] : (int64_t)e * a.cap;
    const int64_t most = a.seg ? a.rows : a.cap;
    *bad = c < 0 || b < 0;
    if (c < 0) c = 0;
    if (b < 0) { b = 0; c = 0; }
    if (c > most) { c = most; *bad = true; }
    if (b > a.rows) { b = a.rows; *bad = *bad || c > 0; }
    if (c > a.rows - b) { c = a.rows - b; *bad = true; }
    *begin = b;
    return c;
}

struct GroupedTile {
    int e;
    int m;                       // row tile of the expert
    int n;                       // column tile
    int64_t begin;               // the expert's first row
    int64_t count;
};

// The number of tiles before the end of every expert, into LDS (ends[L]);
// returns all of them.  Every wave scans, wave 0 writes; the caller
// synchronises.
template <int MT>
__device__ __forceinline__ int32_t grouped_tile_table(const GroupedArgs &a, int tiles_n, int32_t *ends)
{
    const int lane = threadIdx.x & (kWave - 1);
    int32_t base = 0;
    bool any_bad = false;
    for (int e0 = 0; e0 < a.L; e0 += kWave) {
        int32_t c = 0;
        if (e0 + lane < a.L) {
            int64_t b;
            bool bad;
            c = (int32_t)((grouped_rows(a, e0 + lane, &b, &bad) + MT - 1) / MT) * tiles_n;
            any_bad |= bad;
        }
        const int32_t incl = base + wave_inclusive_scan(c);
        if (threadIdx.x < kWave && e0 + lane < a.L) ends[e0 + lane] = incl;
        base = __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    if (blockIdx.x == 0 && __ballot(any_bad) != 0 && threadIdx.x == 0)
        set_status(a.status, a.seg ? CDL_STATUS_ROWS_OVERFLOW : CDL_STATUS_LL_OVERFLOW);
    return base;
}

// Tile `id` of the table: tiles are ordered by expert, then column tile, then
// row tile (the row tiles of one weight tile run side by side, so its second
// reader finds it in a cache).
__device__ __forceinline__ GroupedTile grouped_tile(const GroupedArgs &a, const int32_t *ends, int tiles_n, int32_t id)
{
    const int lane = threadIdx.x & (kWave - 1);
    GroupedTile t;
    t.e = 0;
    for (int e0 = 0; e0 < a.L; e0 += kWave) {
        const bool before = e0 + lane < a.L && ends[e0 + lane] <= id;
        const int n = __popcll(__ballot(before));
        t.e += n;
        if (n < kWave) break;
    }
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    const int32_t from = t.e ? ends[t.e - 1] : 0;
    const int32_t mt = (ends[t.e] - from) / tiles_n, local = id - from;
    t.n = __builtin_amdgcn_readfirstlane(local / mt);
    t.m = __builtin_amdgcn_readfirstlane(local % mt);
    bool bad;
    t.count = grouped_rows(a, t.e, &t.begin, &bad);
    return t;
}

__device__ __forceinline__ i32x8 mx_frag(u32x4 v)
{
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// v_permlane32_swap: the upper 32 lanes of a trade places with the lower 32
// of b.
__device__ __forceinline__ void swap_halves(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// 32 SwiGLU values of one row across a lane and its partner (lane ^ 32): the
// lane holds values 8 b + 4 (lane / 32) + i at h[4 b + i].  Stores the 16
// code bytes and the scale byte of the group.
__device__ __forceinline__ void store_swiglu_group(const float (&h)[16], int lane, bool live, uint8_t *q, uint8_t *s)
{
    // magnitudes as integers: NaNs order above infinity
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t m = __float_as_uint(h[i]) & 0x7FFFFFFFu;
        am = am > m ? am : m;
    }
    uint32_t other = am;
    swap_halves(am, other);
    am = am > other ? am : other;
    const bool nan = am > 0x7F800000u;
    // the smallest b >= 0 with 6 * 2^(b - 127) >= the largest magnitude, as mx_scale_byte
    const int E = (int)(am >> 23);
    int b = E - 2 + ((am & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    b = E == 255 ? 254 : (b < 0 ? 0 : b);
    const float p = __uint_as_float((uint32_t)b << 23);
    uint32_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[8 * j], h[8 * j + 1], p, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[8 * j + 2], h[8 * j + 3], p, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[8 * j + 4], h[8 * j + 5], p, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, h[8 * j + 6], h[8 * j + 7], p, 3);
        c[j] = nan ? 0u : r;
    }
    // lower lane: codes of values 0-3, 8-11 | 16-19, 24-27 in c[0] | c[1];
    // upper: 4-7, 12-15 | 20-23, 28-31.  After the trade the lower lane has
    // both lanes' c[0], the first 8 bytes, the upper both c[1], the last 8.
    swap_halves(c[0], c[1]);
    if (!live) return;
    const u32x2 w = {(c[0] & 0xFFFFu) | (c[1] << 16), (c[0] >> 16) | (c[1] & 0xFFFF0000u)};
    *reinterpret_cast<u32x2 *>(q + (lane >= 32 ? 8 : 0)) = w;
    if (lane < 32) *s = nan ? (uint8_t)255 : (uint8_t)b;
}

// Exchanges that transpose a quad's 4 x 4 words: lane q's v[j] becomes lane
// j's v[q].
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_word(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ void transpose_quad(int lane, uint32_t &v0, uint32_t &v1, uint32_t &v2, uint32_t &v3)
{
    constexpr int kXor1 = 0xB1, kXor2 = 0x4E;          // quad_perm [1,0,3,2], [2,3,0,1]
    const bool odd = lane & 1, high = lane & 2;
    // (every exchange is made by all lanes, the selects follow)
    const uint32_t x0 = dpp_word<kXor1>(v0), x1 = dpp_word<kXor1>(v1);
    const uint32_t x2 = dpp_word<kXor1>(v2), x3 = dpp_word<kXor1>(v3);
    const uint32_t a0 = odd ? x1 : v0, a1 = odd ? v1 : x0, a2 = odd ? x3 : v2, a3 = odd ? v3 : x2;
    const uint32_t y0 = dpp_word<kXor2>(a0), y1 = dpp_word<kXor2>(a1);
    const uint32_t y2 = dpp_word<kXor2>(a2), y3 = dpp_word<kXor2>(a3);
    v0 = high ? y2 : a0;
    v1 = high ? y3 : a1;
    v2 = high ? a2 : y0;
    v3 = high ? a3 : y1;
}

// Two 32 x 32 blocks of products to bf16 rows: lane l has token column l % 32
// of both, weight rows 8 b + 4 (l / 32) + i in [4 b + i].  The halves trade so
// that the lower lanes have block x's 32 columns of their row and the upper
// ones block y's, 4 chunks of 16 bytes; then the lanes of a quad trade so that
// each store writes runs of 64 bytes (one lane's 16 bytes of a row are a
// request of their own otherwise: 131072 rows of 128 experts, K = N = 4096,
// 1307 -> 1274 us).
//   to    the lane's block: its first of 32 rows, at its first column
//   rows, cols  rows and columns of the block that are written
__device__ __forceinline__ void store_blocks_bf16(const f32x16 &x, const f32x16 &y, int lane, uint16_t *to, int rows,
                                                  int cols, int64_t N, bool vector)
{
    uint32_t p[8], q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        q[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
        swap_halves(p[i], q[i]);
    }
    u32x4 v[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) v[b] = u32x4{p[2 * b], p[2 * b + 1], q[2 * b], q[2 * b + 1]};
    const int r = lane & 31;
    if (vector) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t t[4] = {v[0][w], v[1][w], v[2][w], v[3][w]};
            transpose_quad(lane, t[0], t[1], t[2], t[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j][w] = t[j];
        }
        const int c = (lane & 3) * 8, r0 = r & ~3;
        uint16_t *o = to + r0 * N + c;
#pragma unroll
        for (int j = 0; j < 4; ++j, o += N)
            if (r0 + j < rows && c < cols) *reinterpret_cast<u32x4 *>(o) = v[j];
    } else if (r < rows) {
        uint16_t *o = to + r * N;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (8 * b + e < cols) o[8 * b + e] = (uint16_t)(v[b][e / 2] >> (16 * (e & 1)));
    }
}

// Tiles of 256 weight rows (SwiGLU: 128 gate rows and the 128 up rows of the
// same columns) and MT token rows, one at a time per workgroup of 8 waves,
// WN x WM of them; one workgroup per CU takes every 32nd tile of its XCD's
// contiguous eighth (workgroup index mod 8 is the XCD).
//
// Depth stages of 256 elements (128 bytes of a row) pass through two LDS
// buffers: while stage s is multiplied, stage s + 1 goes from registers to
// the other buffer and stage s + 2 is loaded into the registers (8 lanes read
// one row's 128-byte line).  16-byte chunk c of row r lies at chunk
// c ^ (r / 2 % 8), so that 16 consecutive rows touch all 64 banks.
//
// v_mfma_scale_f32_32x32x64: lane l holds row l % 32 of its operand and 32
// consecutive elements of it (16 bytes, one scale byte); D has token column
// l % 32 and, in register i, weight row 8 (i / 4) + 4 (l / 32) + i % 4.  The
// order of the depth is free as long as both operands share it: in a stage's
// four steps the lower 32 lanes take groups 0-3 and the upper ones groups
// 4-7, so a lane's four scale bytes are one aligned word, selected by the
// instruction's byte index.
//
// A wave's order within a stage is fixed by hand: one matrix instruction, then
// a share of the other work (the fragments of the next step, a unit to LDS, the
// load that refills its registers), so that these issue in the shadow of the
// matrix pipe; the barrier stands before the last step, whose fragments are in
// registers by then, and the next stage's first fragments are read under it.
constexpr int kGroupedThreads = 512;
constexpr int kGroupedNT = 256;
constexpr int kGroupedWgs = 256;         // one per CU
constexpr int kStage = 128;              // bytes of a row per stage (256 elements, 8 scales)

template <int MT>
struct GroupedShape {
    static constexpr int WN = MT == 256 ? 2 : 4;
    // wave w has weight part w % WN and token part w / WN: the two waves of a
    // SIMD (w, w + 4) are in different halves of the token rows, so a tile that
    // is half full keeps every SIMD busy
    static constexpr int WM = 8 / WN;
    static constexpr int NF = kGroupedNT / 32 / WN;      // 32-row fragments per wave
    static constexpr int MF = MT / 32 / WM;
    static constexpr int kRows = kGroupedNT + MT;        // LDS rows of a stage
    static constexpr int kUnits = kRows * 8 / kGroupedThreads;   // 16-byte units per thread and stage
    // codes of two stages, the scales of two pairs of stages (16 bytes a row, a row per thread), then the tile table
    static constexpr size_t kLds = 2 * (size_t)kRows * kStage + 2 * (size_t)kGroupedThreads * 16;
};

// The 16 scale bytes of two stages of a row that start at byte `at` of the
// descriptor, from the aligned words that hold them; bytes from `left` on are
// zero.
__device__ __forceinline__ u32x4 pair_scale_bytes(u32x4 v, uint32_t x, uint32_t at, int left)
{
    const uint32_t w[5] = {v.x, v.y, v.z, v.w, x};
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = left - 4 * i;
        const uint32_t keep = n >= 4 ? ~0u : n <= 0 ? 0u : ~0u >> (32 - 8 * n);
        o[i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], at & 3u) & keep;
    }
    return o;
}

template <int MT, bool SWIGLU>
struct GroupedWg {
    using S = GroupedShape<MT>;
    static constexpr int kCols = SWIGLU ? kGroupedNT / 2 : kGroupedNT;     // output columns of a tile
    static constexpr int kBuf = S::kRows * kStage;
    static constexpr uint32_t kFar = 0x80000000u;    // no tile operand reaches this offset
    // Weight rows lie in LDS in blocks of 32, a wave's fragments in order
    // (SwiGLU: its gate fragments, then the up ones of the same columns).
    // Unit j of a thread is 16 bytes of LDS row 64 j + tid / 8, in block
    // 2 j + tid / 256.  With 4 fragments a wave (2 gate, 2 up) units 0 and 2
    // are gate rows and 1 and 3 up rows; with 2 (1 gate, 1 up) the upper half
    // of the threads carries the up rows.
    static constexpr bool kUpByUnit = SWIGLU && S::NF == 4, kUpByHalf = SWIGLU && S::NF == 2;
    static_assert(!SWIGLU || kUpByUnit || kUpByHalf, "fragments per wave");
    const GroupedArgs a;
    uint8_t *const lds;
    const int tid, lane, wave;
    const uint32_t K2;
    const int K32;
    const bool ragged;                       // scale rows not word-aligned
    const uint32_t unit_off, unit_lds;       // a thread's unit 0: operand offset, LDS offset
    const uint32_t scale_lds, scale_lane;    // its scale row's LDS offset; a lane's scale word in a fragment's
    const uint32_t frag_w, frag_b;           // a lane's first fragments: LDS offset at step 0
    // the tile
    int64_t row0, n0;
    int live_m, live_n;
    const uint8_t *w_q, *tok_q, *scale_ptr;  // the wave's first rows
    uint32_t w_bytes, tok_bytes, scale_bytes;
    uint32_t scale_off, sc_off;              // a thread's scale row; that of the scales in registers
    // registers on the way to LDS
    u32x4 stage[S::kUnits];
    u32x4 sc;
    uint32_t sc_x;
    int pair;                                // LDS buffer of the scales stored last
    // A weight fragment is read again for the next step as soon as the last
    // instruction that takes it is issued; the token fragments, which every
    // instruction of a step takes, alternate between two sets.
    f32x16 acc[S::NF][S::MF];
    u32x4 fw[S::NF], fb[2][S::MF];
    int sw[S::NF], sb[S::MF], sb_next[S::MF];   // scale words of a stage

    // LDS row of thread t's scales: waves 0-3 the weight rows, a wave's all
    // gate or all up rows.
    static __device__ __forceinline__ uint32_t scale_row(int t)
    {
        if (!SWIGLU || t >= kGroupedNT) return (uint32_t)t;
        constexpr int H = SWIGLU ? S::NF / 2 : 1;
        const int b = (t & 127) >> 5;
        return (uint32_t)((b / H * S::NF + b % H + (t >= 128 ? H : 0)) * 32 + (t & 31));
    }

    __device__ __forceinline__ GroupedWg(const GroupedArgs &args, uint8_t *l)
        : a(args), lds(l), tid(threadIdx.x), lane(tid & (kWave - 1)), wave(wave_id()), K2((uint32_t)(args.K / 2)),
          K32((int)(args.K / 32)),
          ragged((((uint32_t)K32 | (uint32_t)(uintptr_t)args.s | (uint32_t)(uintptr_t)args.ws) & 3u) != 0),
          unit_off((uint32_t)(tid >> 3) % 32 * K2 + (uint32_t)(tid & 7) * 16),
          unit_lds((uint32_t)(tid >> 3) * kStage + (uint32_t)(((tid & 7) ^ (tid >> 4 & 7)) << 4)),
          scale_lds(2 * kBuf + scale_row(tid) * 16),
          scale_lane((uint32_t)((lane & 31) * 16 + (lane >> 5) * 4)),
          frag_w((uint32_t)((wave % S::WN) * S::NF * 32 + (lane & 31)) * kStage +
                 (uint32_t)(((4 * (lane >> 5)) ^ (lane >> 1 & 7)) << 4)),
          frag_b((uint32_t)(kGroupedNT + (wave / S::WN) * S::MF * 32 + (lane & 31)) * kStage +
                 (uint32_t)(((4 * (lane >> 5)) ^ (lane >> 1 & 7)) << 4))
    {
    }

    __device__ __forceinline__ void set_tile(const GroupedTile &t)
    {
        const int64_t I = a.N / 2, m0 = (int64_t)t.m * MT, n_rows = SWIGLU ? I : a.N;
        n0 = (int64_t)t.n * kCols;
        row0 = t.begin + m0;
        live_m = (int)(t.count - m0 < MT ? t.count - m0 : MT);
        live_n = (int)(n_rows - n0 < kCols ? n_rows - n0 : kCols);
        const int skip = wave / 4 * 32;      // rows of the wave's first unit
        const int64_t w_row = (int64_t)t.e * a.N + n0;
        const int left_m = live_m > skip ? live_m - skip : 0;
        tok_q = a.q + (row0 + skip) * K2;
        tok_bytes = (uint32_t)left_m * K2;
        if (kUpByHalf) {
            w_q = a.wq + (w_row + (wave >= 4 ? I : 0)) * K2;
            w_bytes = (uint32_t)live_n * K2;
        } else {
            w_q = a.wq + (w_row + skip) * K2;
            w_bytes = (uint32_t)(live_n > skip ? live_n - skip : 0) * K2;
        }
        // Scale rows start at any byte: the descriptor begins at the word
        // below and ends with the word that holds the last byte.
        const uint8_t *sp;
        uint32_t rows, in;
        if (wave < kGroupedNT / kWave) {
            sp = a.ws + (w_row + (SWIGLU && wave >= 2 ? I : 0)) * K32;
            rows = (uint32_t)live_n;
            in = (uint32_t)(SWIGLU ? tid & 127 : tid);
        } else {
            sp = a.s + row0 * K32;
            rows = (uint32_t)live_m;
            in = (uint32_t)(tid - kGroupedNT);    // at or past live_m: out of range
        }
        const uint32_t shift = (uint32_t)(uintptr_t)sp & 3u;
        scale_ptr = sp - shift;
        scale_bytes = (shift + rows * (uint32_t)K32 + 3) & ~3u;
        scale_off = shift + in * (uint32_t)K32;
    }

    // No tile to load: every operand is empty.
    __device__ __forceinline__ void set_no_tile() { w_bytes = tok_bytes = scale_bytes = 0; }

    // A thread's offset into stage s of its rows: past the row's end (also
    // for whole stages past the last) beyond every operand, where loads read
    // no memory and return zeros.
    __device__ __forceinline__ uint32_t stage_off(int s) const
    {
        const uint32_t k = (uint32_t)s * kStage;
        return k + ((uint32_t)tid & 7) * 16 < K2 ? unit_off + k : kFar;
    }
    // unit j of a stage; *off is unit 0's offset for j = 0 and advances
    __device__ __forceinline__ void load_unit(uint32_t *off, uint32_t off0, int j)
    {
        constexpr int kWeightUnits = kGroupedNT / 64;
        if (j == kWeightUnits) *off = off0;
        if (j < kWeightUnits) {
            const uint8_t *p = w_q;
            if (kUpByUnit && j % 2 == 1) p += a.N / 2 * K2;
            stage[j] = buf_ld16(make_rsrc(p, w_bytes), *off, 0);
            if (!kUpByUnit || j % 2 == 1) *off += (kUpByHalf ? 32 : 64) * K2;
        } else {
            stage[j] = buf_ld16(make_rsrc(tok_q, tok_bytes), *off, 0);
            *off += 64 * K2;
        }
    }
    __device__ __forceinline__ void store_unit(int buf, int j)
    {
        *reinterpret_cast<u32x4 *>(lds + (unit_lds + (uint32_t)(buf * kBuf)) + j * (64 * kStage)) = stage[j];
    }
    // The scales of stages s and s + 1 (s even), one row a thread (threads past
    // the rows: zeros): every row is a cache line of its own, so that a load
    // for each stage costs as much as the codes' (decode 95 -> 86 us, 4096
    // rows of 32 experts 135 -> 126 us by taking two stages at once).
    __device__ __forceinline__ void load_scales(int s)
    {
        const rsrc_t r = make_rsrc(scale_ptr, scale_bytes);
        const uint32_t at = (scale_off + 8u * (uint32_t)s) & ~3u;
        sc_off = scale_off;
        sc = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
        sc_x = ragged ? (uint32_t)buf_ld4(r, at + 16u, 0) : 0u;
    }
    __device__ __forceinline__ void store_scales(int s)
    {
        pair ^= 1;
        *reinterpret_cast<u32x4 *>(lds + scale_lds + pair * (kGroupedThreads * 16)) =
            pair_scale_bytes(sc, sc_x, sc_off, K32 - 8 * s);
    }

    // fragments of step `st` of the stage in LDS buffer buf
    __device__ __forceinline__ u32x4 weight_fragment(int buf, int st, int n) const
    {
        return *reinterpret_cast<const u32x4 *>(lds + ((frag_w ^ (uint32_t)(st << 4)) + (uint32_t)(buf * kBuf)) +
                                                n * (32 * kStage));
    }
    __device__ __forceinline__ u32x4 token_fragment(int buf, int st, int m) const
    {
        return *reinterpret_cast<const u32x4 *>(lds + ((frag_b ^ (uint32_t)(st << 4)) + (uint32_t)(buf * kBuf)) +
                                                m * (32 * kStage));
    }
    // scale words of stage s of a tile, whose pair was stored last
    __device__ __forceinline__ uint32_t pair_scales(int s) const
    {
        return 2 * kBuf + (uint32_t)(pair * (kGroupedThreads * 16) + (s & 1) * 8) + scale_lane;
    }
    __device__ __forceinline__ int weight_scale(int s, int n) const
    {
        return *reinterpret_cast<const int *>(lds + pair_scales(s) + wave % S::WN * (S::NF * 512) + n * 512);
    }
    __device__ __forceinline__ int token_scale(int s, int m) const
    {
        return *reinterpret_cast<const int *>(lds + pair_scales(s) + wave / S::WN * (S::MF * 512) +
                                              (kGroupedNT / 32 + m) * 512);
    }

    // Share of `total` items that follows matrix instruction i of `of`.
    template <typename F>
    static __device__ __forceinline__ void share(int i, int of, int total, F &&f)
    {
#pragma unroll
        for (int x = 0; x < total; ++x)
            if (x * of / total == i) f(x);
    }

    // Step ST of the stage in LDS buffer buf: its matrix instructions, each
    // followed by the reads for the next step (after the last, of stage `next`
    // of its tile) and by work(i).
    template <int ST, typename F>
    __device__ __forceinline__ void multiply(int buf, int next, F &&work)
    {
        constexpr int NM = S::NF * S::MF, SET = ST & 1, nst = (ST + 1) & 3;
        const int nbuf = ST == 3 ? buf ^ 1 : buf;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            const int n = i / S::MF, m = i % S::MF;
            acc[n][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_frag(fw[n]), mx_frag(fb[SET][m]), acc[n][m],
                                                                        4, 4, ST, sw[n], ST, sb[m]);
            __builtin_amdgcn_sched_barrier(0);
            share(i, NM, S::MF, [&](int x) {
                fb[SET ^ 1][x] = token_fragment(nbuf, nst, x);
                if (ST == 3) sb_next[x] = token_scale(next, x);
            });
            if (m == S::MF - 1) {
                fw[n] = weight_fragment(nbuf, nst, n);
                if (ST == 3) sw[n] = weight_scale(next, n);
            }
            work(i);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // One stage of the tile, in LDS buffer buf, its first fragments and scales
    // in registers; leaves the next stage's there.  The registers hold stage
    // `held` of its tile, which goes to the other buffer, and take stage
    // `load` of the tile set last.
    template <bool BUSY>
    __device__ __forceinline__ void run_stage(int buf, int held, int load)
    {
        constexpr int NM = S::NF * S::MF, U = S::kUnits;
        const uint32_t off0 = stage_off(load);
        uint32_t off = off0;
        auto refill = [&](int x) {
            store_unit(buf ^ 1, x);
            load_unit(&off, off0, x);
        };
        if (!(held & 1)) store_scales(held);
        if (!(load & 1)) load_scales(load);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (BUSY) {
            multiply<0>(buf, held, [&](int i) { share(i, 2 * NM, U, refill); });
            multiply<1>(buf, held, [&](int i) { share(i + NM, 2 * NM, U, refill); });
            multiply<2>(buf, held, [&](int) {});
            __syncthreads();
            multiply<3>(buf, held, [&](int) {});
#pragma unroll
            for (int j = 0; j < S::MF; ++j) sb[j] = sb_next[j];
        } else {
#pragma unroll
            for (int x = 0; x < U; ++x) refill(x);
            __syncthreads();
        }
    }

    // Before the first tile: its stage 0 to LDS buffer 0, stage 1 to the
    // registers.
    __device__ __forceinline__ void start()
    {
        uint32_t off0 = stage_off(0), off = off0;
#pragma unroll
        for (int j = 0; j < S::kUnits; ++j) load_unit(&off, off0, j);
        load_scales(0);
        off0 = stage_off(1);
        off = off0;
#pragma unroll
        for (int j = 0; j < S::kUnits; ++j) {
            store_unit(0, j);
            load_unit(&off, off0, j);
        }
        pair = 1;
        store_scales(0);
        __syncthreads();
    }

    // A tile's products into acc.  Its first stage is in LDS buffer buf, the
    // second in registers; leaves the next tile's there (set by next(), called
    // before the last two stages, which load for it).  stages >= 2.
    template <bool BUSY, typename F>
    __device__ __forceinline__ int run_tile(int buf, int stages, F &&next)
    {
        if constexpr (BUSY) {
#pragma unroll
            for (int i = 0; i < S::NF; ++i) {
                sw[i] = weight_scale(0, i);
                fw[i] = weight_fragment(buf, 0, i);
#pragma unroll
                for (int j = 0; j < S::MF; ++j) acc[i][j] = f32x16{};
            }
#pragma unroll
            for (int j = 0; j < S::MF; ++j) {
                sb[j] = token_scale(0, j);
                fb[0][j] = token_fragment(buf, 0, j);
            }
        }
        for (int s = 0; s < stages; ++s) {
            const int ahead = s + 2 - stages;
            if (ahead == 0) next();
            run_stage<BUSY>(buf, ahead == 1 ? 0 : s + 1, ahead >= 0 ? ahead : s + 2);
            buf ^= 1;
        }
        return buf;
    }

    __device__ __forceinline__ void store_tile(int64_t row_first, int64_t n_first, int rows_m, int cols)
    {
        const int wn = wave % S::WN, wm = wave / S::WN;
        if constexpr (SWIGLU) {
            constexpr int H = S::NF / 2;
            const int64_t I = a.N / 2;
#pragma unroll
            for (int j = 0; j < S::MF; ++j) {
                const int m = (wm * S::MF + j) * 32 + (lane & 31);
                const int64_t row = row_first + m;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int n = (wn * H + i) * 32;
                    if (n >= cols) continue;
                    float h[16];
#pragma unroll
                    for (int v = 0; v < 16; ++v) h[v] = acc[i][j][v] / (1.0f + __expf(-acc[i][j][v])) * acc[i + H][j][v];
                    store_swiglu_group(h, lane, m < rows_m, a.hq + row * (I / 2) + (n_first + n) / 2,
                                       a.hs + row * (I / 32) + (n_first + n) / 32);
                }
            }
        } else {
            const bool vector = a.N % 8 == 0 && ((uintptr_t)a.out & 15) == 0;      // rows keep the 16-byte alignment
            // pairs of blocks: both token fragments of a weight fragment, or
            // (one token fragment) two weight fragments
            constexpr int P = S::MF == 2 ? S::NF : S::NF / 2;
            static_assert(S::MF == 2 || S::MF == 1, "token fragments per wave");
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int up = lane >> 5;
                const int n = (wn * S::NF + (S::MF == 2 ? i : 2 * i + up)) * 32;
                const int m = (wm * S::MF + (S::MF == 2 ? up : 0)) * 32;
                store_blocks_bf16(acc[S::MF == 2 ? i : 2 * i][0], S::MF == 2 ? acc[i][1 % S::MF] : acc[(2 * i + 1) % S::NF][0],
                                  lane, a.out + (row_first + m) * a.N + n_first + n, rows_m - m, cols - n, a.N, vector);
                __builtin_amdgcn_sched_barrier(0);     // one pair's temporaries at a time
            }
        }
    }
};

template <int MT, bool SWIGLU>
__global__ __launch_bounds__(kGroupedThreads) void grouped_kernel(GroupedArgs a, int tiles_n)
{
    using Wg = GroupedWg<MT, SWIGLU>;
    using S = GroupedShape<MT>;
    extern __shared__ u32x4 lds4[];
    uint8_t *lds = reinterpret_cast<uint8_t *>(lds4);
    int32_t *ends = reinterpret_cast<int32_t *>(lds + S::kLds);
    const int32_t total = grouped_tile_table<MT>(a, tiles_n, ends);
    const int32_t per = (total + 7) / 8, step = (int32_t)(gridDim.x / 8);
    const int32_t first = (int32_t)(blockIdx.x & 7) * per;
    const int32_t last = first + per < total ? first + per : total;
    int32_t id = first + (int32_t)(blockIdx.x >> 3);
    if (id >= last) return;
    __syncthreads();
    // two at least (an empty one reads no memory): the last two load the next tile's first
    const int stages = a.K > 256 ? (int)((a.K / 2 + kStage - 1) / kStage) : 2;
    Wg w(a, lds);
    w.set_tile(grouped_tile(a, ends, tiles_n, id));
    w.start();
    for (int buf = 0;;) {
        const int64_t row0 = w.row0, n0 = w.n0;
        const int live_m = w.live_m, live_n = w.live_n;
        const bool busy = w.wave / S::WN * S::MF * 32 < live_m;      // the wave has a live token column
        id += step;
        auto next = [&] {
            if (id < last)
                w.set_tile(grouped_tile(a, ends, tiles_n, id));
            else
                w.set_no_tile();
        };
        buf = busy ? w.template run_tile<true>(buf, stages, next) : w.template run_tile<false>(buf, stages, next);
        if (busy) w.store_tile(row0, n0, live_m, live_n);
        if (id >= last) return;
    }
}

// ---------------------------------------------------------------------------
// the MoE layer of a few tokens
// ---------------------------------------------------------------------------

constexpr int kFewThreads = 256;        // first kernel: 4 waves share the columns, split the depth
constexpr int kFewWaves = kFewThreads / kWave;
constexpr int kFewMaxSlots = 4096;

struct FewArgs {
    const uint16_t *x;           // [T, H]
    const int32_t *ids;
    const float *weights;        // [T, k]
    int32_t T, k, expert_begin, L;
    int64_t H, I;
    const uint8_t *w13, *w13_s;  // [L, 2 I, H] bf16, or MXFP4 bytes and scales
    const uint8_t *w2, *w2_s;    // [L, H, I]
    uint16_t *out;               // [T, H]
    int32_t *lists;              // see FewLists
    uint16_t *h;                 // [T k, I], twice for up to kSplitTokens tokens
};

// The activations between the products are rounded to bf16, the second
// product's operand type (error against 64 bits 0.0024, of which 0.0017 is the
// output's own rounding; the remainder for every batch took 128 tokens of 32 of
// 256 experts from 480 to 519 us).  Up to two tokens use 2 of its 16 columns:
// there the rounding's remainder takes two more, at the price of a row load a
// turn (one token, H = 7168, I = 2048, top-8: 44 us with either in MXFP4).
constexpr int kSplitTokens = 2;
constexpr int kSplitXt = 1;                     // the first kernel's column loads for them

// Up to 64 slots, the routing lists hold the experts with slots in the order
// of their first slot; above, all L experts.
__host__ __device__ inline int few_experts(int n, int L) { return n > kWave ? L : n < L ? n : L; }

// Routing lists in the workspace, written by the first kernel: the number of
// experts listed, then for the a-th of them its index and the begin of its
// slots, then the slots (flat t * k + j, ascending within an expert).
struct FewLists {
    int32_t *active, *expert, *begin, *slots;
    __host__ __device__ FewLists(int32_t *p, int A) : active(p), expert(p + 4), begin(p + 4 + A), slots(p + 4 + 2 * A + 4) {}
    static size_t ints(int64_t A, int64_t n) { return (size_t)(4 + A + A + 4 + n); }
};

template <int STEP>
__device__ __forceinline__ v8bf16 few_expand(u32x4 w, float p)
{
    const uint32_t c = STEP == 0 ? w.x : STEP == 1 ? w.y : STEP == 2 ? w.z : w.w;
    const u32x4 r = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, p, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, p, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, p, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, p, 3))};
    return __builtin_bit_cast(v8bf16, r);
}

// 16 rows of weights through descriptors of their own (zeros past them).
// MXFP4 scale rows start at any byte: their descriptor begins at the word
// below (`shift` bytes before) and ends with the word that holds the last one.
template <bool FP4>
struct FewRows {
    rsrc_t q, s;
    uint32_t shift;
    __device__ __forceinline__ FewRows() {}
    __device__ __forceinline__ FewRows(const uint8_t *w, const uint8_t *ws, int64_t row, int64_t rows, int64_t depth)
    {
        if (rows < 0) rows = 0;
        if constexpr (FP4) {
            q = make_rsrc(w + row * (depth / 2), (uint32_t)(rows * (depth / 2)));
            const uint8_t *sp = ws + row * (depth / 32);
            shift = (uint32_t)(uintptr_t)sp & 3u;
            s = make_rsrc(sp - shift, rows ? (uint32_t)(shift + rows * (depth / 32) + 3) & ~3u : 0u);
        } else {
            q = make_rsrc(w + row * depth * 2, (uint32_t)(rows * depth * 2));
            shift = 0;
        }
    }
};

// The depth is taken in turns of 256 elements.  v_mfma_f32_16x16x32_bf16: lane
// l holds row (column) l % 16 of its operand and 8 consecutive elements; the
// order of the depth is free as long as both operands share it.  bf16: step i
// of a turn is elements 32 i + 8 (l / 16) on, one 16-byte load per 16 rows.
// MXFP4: a lane's 16 bytes are one group of 32 elements, which serve 4
// instructions; step i (of 2) of a turn is group 2 (l / 16) + i, so that a
// lane's two scale bytes are neighbours and arrive in one load.
constexpr uint32_t kTurn = 256;

// The weights of G steps of NW blocks of 16 rows.
template <bool FP4, int NW, int G>
struct FewWeights {
    static_assert(!FP4 || G == 2, "a turn of MXFP4 weights is two steps");
    u32x4 w[G][NW];
    u32x2 s[NW];
    uint32_t at[NW];                           // byte of the lane's first scale in its words, at % 4

    // steps from `first` on of the turn at element d; past `depth` no memory is read
    template <bool SCALES>
    __device__ __forceinline__ void load(const FewRows<FP4> (&rows)[NW], uint32_t depth, uint32_t d, int first)
    {
        const uint32_t lane = threadIdx.x & (kWave - 1), r = lane & 15, g = lane >> 4;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const uint32_t at = FP4 ? d + (2 * g + j) * 32 : d + (first + j) * 32 + g * 8;
            const uint32_t off = at < depth ? (FP4 ? r * (depth / 2) + at / 2 : (r * depth + at) * 2) : 0xFFFFFFF0u;
#pragma unroll
            for (int n = 0; n < NW; ++n) w[j][n] = buf_ld16(rows[n].q, off, 0);
        }
        if constexpr (FP4 && SCALES) {
#pragma unroll
            for (int n = 0; n < NW; ++n) {
                at[n] = rows[n].shift + r * (depth / 32) + d / 32 + 2 * g;
                s[n] = __builtin_amdgcn_raw_buffer_load_b64(rows[n].s, at[n] & ~3u, 0, 0);
            }
        }
    }
    // the lane's two scale bytes of block n
    __device__ __forceinline__ uint32_t scales(int n) const { return __builtin_amdgcn_alignbyte(s[n].y, s[n].x, at[n] & 3u); }
    // acc[n] += block n * columns; column(chunk) is the lane's column's 8
    // elements from 8 chunk on of the turn, scale(n) the lane's two scale bytes
    // of block n
    template <typename F, typename S>
    __device__ __forceinline__ void multiply(f32x4 (&acc)[NW], uint32_t depth, uint32_t d, int first, F &&column, S &&scale)
    {
        const uint32_t lane = threadIdx.x & (kWave - 1), g = lane >> 4;
        if constexpr (FP4) {
            uint32_t bytes[NW];
#pragma unroll
            for (int n = 0; n < NW; ++n) bytes[n] = scale(n);
#pragma unroll
            for (int j = 0; j < G; ++j) {
                v8bf16 b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = column((2 * g + j) * 4 + i);
                const bool in = d + (2 * g + j) * 32 < depth;
                float p[NW];
#pragma unroll
                for (int n = 0; n < NW; ++n) {
                    // (past the depth: codes and scale zero)
                    p[n] = __uint_as_float(in ? (bytes[n] >> (8 * j) & 0xFFu) << 23 : 0u);
                }
                auto part = [&](auto c) {
                    constexpr int st = decltype(c)::value;
#pragma unroll
                    for (int n = 0; n < NW; ++n)
                        acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_expand<st>(w[j][n], p[n]), b[st], acc[n], 0, 0, 0);
                };
                part(std::integral_constant<int, 0>{});
                part(std::integral_constant<int, 1>{});
                part(std::integral_constant<int, 2>{});
                part(std::integral_constant<int, 3>{});
            }
        } else {
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const v8bf16 b = column((first + j) * 4 + g);
#pragma unroll
                for (int n = 0; n < NW; ++n)
                    acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf16, w[j][n]), b, acc[n], 0, 0, 0);
            }
        }
    }
};

// A turn of up to 2 XT bf16 rows, the columns of the product, on its way
// through a wave's own 2 XT x 512 bytes of LDS: a load brings two rows (32 lanes
// of 16 bytes each), where fragments straight from memory would take a load
// of 64 lanes for every 32 elements whatever the number of rows.  16-byte
// chunk q of row r lies at q ^ r.
template <int XT>
struct FewColumns {
    u32x4 v[XT];
    uint8_t *lds;

    // row_off(i): byte offset of row i; elements past `depth` are zero
    template <typename F>
    __device__ __forceinline__ void load(rsrc_t r, uint32_t depth, uint32_t d, F &&row_off)
    {
        const uint32_t lane = threadIdx.x & (kWave - 1), at = d + (lane & 31) * 8;
#pragma unroll
        for (int j = 0; j < XT; ++j) {
            const uint32_t off = row_off(2 * j + (int)(lane >> 5)) + at * 2;
            v[j] = buf_ld16(r, at < depth ? off : 0xFFFFFFF0u, 0);
        }
    }
    __device__ __forceinline__ void store() const
    {
        const uint32_t lane = threadIdx.x & (kWave - 1), q = lane & 31;
#pragma unroll
        for (int j = 0; j < XT; ++j) {
            const uint32_t r = 2 * j + (lane >> 5);
            *reinterpret_cast<u32x4 *>(lds + r * 512 + ((q ^ r) << 4)) = v[j];
        }
    }
    // the lane's column (rows from 2 XT on repeat the first ones: unused columns)
    __device__ __forceinline__ v8bf16 chunk(uint32_t q) const
    {
        const uint32_t r = (threadIdx.x & 15) & (2 * XT - 1);
        return *reinterpret_cast<const v8bf16 *>(lds + r * 512 + ((q ^ r) << 4));
    }
};

// First kernel: h[slot, i] = silu(gate) * up for 16 columns i of the a-th
// listed expert (blockIdx.y); blockIdx.x is the column tile.  The 4 waves take
// the turns of the depth in rotation, a part of a turn being multiplied while
// the next one arrives, and add their sums in LDS.  LDS_SCALES: MXFP4 scales
// of the whole depth lie in LDS.
template <bool FP4, int XT, bool LDS_SCALES>
__global__ __launch_bounds__(kFewThreads, 2) void few_gate_up_kernel(FewArgs a)
{
    constexpr int NW = 2, kSlots = 2 * XT;     // a gate and an up block; slots at a time
    constexpr int G = FP4 ? 2 : 4;
    extern __shared__ u32x4 lds4[];
    int16_t *list = reinterpret_cast<int16_t *>(lds4);             // [n] the expert's slots (n > 64)
    __shared__ f32x4 part[kFewWaves][NW][kWave];
    __shared__ u32x4 columns[kFewWaves][kSlots * 512 / 16];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    const int n = a.T * a.k;
    const FewLists ls(a.lists, few_experts(n, a.L));
    // every expert's first workgroup writes the expert's own list
    const bool publish = blockIdx.x == 0 && wave == 0;
    int mine = -1, count = 0, before = 0, one_slot = 0;
    const int c = lane & 15, g = lane >> 4;
    const uint32_t H = (uint32_t)a.H;
    const int64_t i0 = (int64_t)blockIdx.x * 16;
    const int64_t live_i = a.I - i0 < 16 ? a.I - i0 : 16;
    constexpr bool kLdsScales = FP4 && LDS_SCALES;
    FewRows<FP4> rows[NW];
    FewWeights<FP4, NW, G> w[2];
    auto set_rows = [&] {
        mine = __builtin_amdgcn_readfirstlane(mine);
#pragma unroll
        for (int i = 0; i < NW; ++i)
            rows[i] = FewRows<FP4>(a.w13, a.w13_s, (int64_t)mine * 2 * a.I + i * a.I + i0, live_i, a.H);
    };
    auto load_w = [&](FewWeights<FP4, NW, G> &t, uint32_t at, int first) {
        t.template load<!kLdsScales>(rows, H, at, first);
    };
    bool ahead = false;                        // the first weights are on their way
    // every wave finds the expert's slots by itself
    if (n <= kWave) {
        // slot i lies in lane i
        const int e = lane < n ? local_expert(a.ids[lane], a.expert_begin, a.L) : -1;
        uint64_t left = __ballot(e >= 0), mask = 0;
        int a_th = 0;
        while (left) {
            const int el = __builtin_amdgcn_readlane(e, (int)__builtin_ctzll(left));
            const uint64_t m = __ballot(e == el);
            if (a_th == (int)blockIdx.y) {
                mine = el;
                mask = m;
            }
            if (a_th < (int)blockIdx.y) before += __popcll(m);
            ++a_th;
            left &= ~m;
        }
        count = __popcll(mask);
        if (publish && lane == 0 && blockIdx.y == 0) ls.active[0] = a_th;
        if (publish && (mask >> lane & 1)) ls.slots[before + __popcll(mask & lanes_below(lane))] = lane;
        // lane i takes the expert's i-th slot
        int at = 0;
        for (uint64_t m = mask; m; m &= m - 1, ++at) {
            const int slot = (int)__builtin_ctzll(m);
            if (at == lane) one_slot = slot;
        }
    } else {
        // the expert is known: its first weights are loaded behind the first ids
        // where there are slots for most experts
        mine = (int)blockIdx.y;
        constexpr int kBatch = 8;
        int32_t id[kBatch];
        auto load_ids = [&](int s0) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int i = s0 + q * kWave + lane;
                id[q] = a.ids[i < n ? i : 0];
            }
        };
        load_ids(0);
        set_rows();
        ahead = n >= a.L;
        if (ahead) load_w(w[0], (uint32_t)wave * kTurn, 0);
        // all waves write the same list
        for (int s0 = 0; s0 < n; s0 += kBatch * kWave) {
            if (s0) load_ids(s0);
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int i = s0 + q * kWave + lane;
                const int e = i < n ? local_expert(id[q], a.expert_begin, a.L) : -1;
                const uint64_t m = __ballot(e == mine);
                if (e == mine) {
                    const int to = count + __popcll(m & lanes_below(lane));
                    list[to] = (int16_t)i;
                }
                count += __popcll(m);
                before += __popcll(__ballot(e >= 0 && e < mine));
            }
        }
        if (publish) {
            if (lane == 0 && blockIdx.y == 0) ls.active[0] = a.L;
            for (int i = lane; i < count; i += kWave) ls.slots[before + i] = list[i];
        }
    }
    if (publish && lane == 0 && mine >= 0) {
        ls.expert[blockIdx.y] = mine;
        ls.begin[blockIdx.y] = before;
        ls.begin[blockIdx.y + 1] = before + count;
    }
    if (count == 0) return;
    if (n <= kWave) set_rows();
    const rsrc_t xr = make_rsrc(a.x, (uint32_t)(a.T * a.H * 2));
    // The scales of a block's 16 rows are one run of bytes: they are brought to
    // LDS whole, where a load per turn would fetch every row's line again.
    uint8_t *scales = reinterpret_cast<uint8_t *>(lds4) + (n > kWave ? (n * 2 + 15) / 16 * 16 : 0);
    const uint32_t run = H / 2, pitch = (run + 3 + 3) & ~3u;       // bytes of a run, and with its first word's shift
    auto slot_of = [&](int i) {                // the expert's i-th slot
        return n <= kWave ? __shfl(one_slot, i, kWave) : (int)list[i];
    };
    for (int c0 = 0; c0 < count; c0 += kSlots) {
        const int live = count - c0 < kSlots ? count - c0 : kSlots;
        const int slot = slot_of(c0 + (c < live ? c : 0));
        f32x4 acc[NW] = {};
        {
            FewColumns<XT> x;
            x.lds = reinterpret_cast<uint8_t *>(columns[wave]);
            uint32_t off[XT];
#pragma unroll
            for (int j = 0; j < XT; ++j) {
                const int i = 2 * j + (lane >> 5);
                off[j] = (uint32_t)(slot_of(c0 + (i < live ? i : 0)) / a.k) * H * 2;
            }
            auto load_x = [&](uint32_t d) { x.load(xr, H, d, [&](int i) { return off[i / 2]; }); };
            auto column = [&](uint32_t q) { return x.chunk(q); };
            auto multiply = [&](FewWeights<FP4, NW, G> &t, uint32_t at, int first) {
                t.multiply(acc, H, at, first, column, [&](int b) -> uint32_t {
                    if constexpr (!kLdsScales) return t.scales(b);
                    // (a turn's last groups may lie past the row's end: read, not used)
                    const uint8_t *p = scales + b * pitch + rows[b].shift + c * (H / 32) + (at < H ? at / 32 + 2 * g : 0);
                    return (uint32_t)p[0] | (uint32_t)p[1] << 8;
                });
            };
            constexpr uint32_t kNext = kTurn * kFewWaves;
            uint32_t d = (uint32_t)wave * kTurn;
            load_x(d);
            if (c0 || !ahead) load_w(w[0], d, 0);
            if constexpr (kLdsScales) {
                if (c0 == 0) {
                    for (uint32_t i = (uint32_t)tid * 4; i < pitch; i += kFewThreads * 4)
#pragma unroll
                        for (int b = 0; b < NW; ++b)
                            *reinterpret_cast<int32_t *>(scales + b * pitch + i) = buf_ld4(rows[b].s, i, 0);
                    __syncthreads();
                }
            }
            x.store();
            load_x(d + kNext);
            if constexpr (FP4) {
                // a part is a turn
                for (; d < H; d += 2 * kNext) {
                    load_w(w[1], d + kNext, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply(w[0], d, 0);
                    x.store();
                    load_x(d + 2 * kNext);
                    __builtin_amdgcn_sched_barrier(0);
                    load_w(w[0], d + 2 * kNext, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply(w[1], d + kNext, 0);
                    x.store();
                    load_x(d + 3 * kNext);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                // a part is half a turn
                for (; d < H; d += kNext) {
                    load_w(w[1], d, 4);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply(w[0], d, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    load_w(w[0], d + kNext, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply(w[1], d, 4);
                    x.store();
                    load_x(d + 2 * kNext);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        if (c0) __syncthreads();               // the sums of the round before are read
#pragma unroll
        for (int i = 0; i < NW; ++i) part[wave][i][lane] = acc[i];
        __syncthreads();
        if (wave == 0) {
            f32x4 gate = part[0][0][lane], up = part[0][1][lane];
#pragma unroll
            for (int w = 1; w < kFewWaves; ++w) {
                gate += part[w][0][lane];
                up += part[w][1][lane];
            }
            if (c < live && 4 * g < live_i) {
                float h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = gate[i] / (1.0f + __expf(-gate[i])) * up[i];
                const u32x2 hi = {pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3])};
                uint16_t *to = a.h + (int64_t)slot * a.I + i0 + 4 * g;
                *reinterpret_cast<u32x2 *>(to) = hi;
                if constexpr (kSplitXt == XT) {
                    // what the rounding left (a non-finite value leaves nothing)
                    float lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = i < 2 ? hi.x : hi.y;
                        const float r = i & 1 ? bf16_hi(w) : bf16_lo(w);
                        lo[i] = __builtin_isfinite(r) ? h[i] - r : 0.0f;
                    }
                    *reinterpret_cast<u32x2 *>(to + (int64_t)n * a.I) = u32x2{pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3])};
                }
            }
        }
    }
}

// Second kernel: out[t, n] for 16 columns n and every token.  The items (an
// expert, a part of its depth) are dealt to the waves in rotation and taken
// 8 slots at a time, turn by turn, the operands of the next turns (two of
// MXFP4, one of bf16) arriving while one is multiplied; each wave adds its weighted products into sums of
// its own in LDS, which are added in wave order.  LDS: the sums, the waves'
// columns, then the lists.
constexpr int kItemSlots = 8;
struct FewDownLds {
    size_t columns, wts, slots, expert, begin, bytes;
    __host__ __device__ FewDownLds(int waves, int T, int n, int A)
    {
        columns = (size_t)waves * T * 64;
        wts = columns + (size_t)waves * kItemSlots * 512;
        slots = wts + (size_t)n * 4;
        expert = slots + (size_t)(n + (n & 1)) * 2;
        begin = expert + (size_t)(A + (A & 1)) * 2;
        bytes = begin + (size_t)(A + 1) * 2;
    }
};

template <bool FP4, int WAVES, bool SPLIT>
__global__ __launch_bounds__(WAVES *kWave) void few_down_kernel(FewArgs a)
{
    constexpr int kSlots = SPLIT ? kSplitTokens : kItemSlots;      // slots at a time
    constexpr int G = FP4 ? 2 : 8;             // a turn
    extern __shared__ u32x4 lds4[];
    uint8_t *lds = reinterpret_cast<uint8_t *>(lds4);
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    const int n = a.T * a.k, A = few_experts(n, a.L);
    const FewLists ls(a.lists, A);
    const FewDownLds at(WAVES, a.T, n, A);
    float *sums = reinterpret_cast<float *>(lds);                          // [waves][T][16]
    float *wts = reinterpret_cast<float *>(lds + at.wts);                  // [n]
    int16_t *slots = reinterpret_cast<int16_t *>(lds + at.slots);          // [n]
    int16_t *expert = reinterpret_cast<int16_t *>(lds + at.expert);        // [A]
    int16_t *begin = reinterpret_cast<int16_t *>(lds + at.begin);          // [A + 1]
    const int active = ls.active[0];
    for (int i = tid; i < n; i += WAVES * kWave) {
        wts[i] = a.weights[i];
        slots[i] = (int16_t)ls.slots[i];       // those behind the last one are not used
    }
    for (int i = tid; i <= A; i += WAVES * kWave) {
        if (i < A) expert[i] = (int16_t)ls.expert[i];
        begin[i] = (int16_t)ls.begin[i];
    }
    float *mine = sums + (size_t)wave * a.T * 16;
    for (int i = lane; i < a.T * 16; i += kWave) mine[i] = 0.0f;
    __syncthreads();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t rows_n = a.H - n0 < 16 ? a.H - n0 : 16;
    const uint32_t I = (uint32_t)a.I;
    int with_slots = 0;
    bool many = false;                         // an expert with more than 2
    for (int i0 = 0; i0 < active; i0 += kWave) {
        const int have = i0 + lane < active ? begin[i0 + lane + 1] - begin[i0 + lane] : 0;
        with_slots += __popcll(__ballot(have > 0));
        many |= __ballot(have > 2) != 0;
    }
    // four items a wave where the experts with slots are few
    const int turns = (int)((I + kTurn - 1) / kTurn);
    int parts = with_slots > 0 ? (4 * WAVES + with_slots - 1) / with_slots : 1;
    parts = parts < turns ? parts : turns;
    const int items = active * parts;
    const int c = lane & 15, g = lane >> 4;
    const rsrc_t hr = make_rsrc(a.h, (uint32_t)n * I * (SPLIT ? 4 : 2));

    auto run = [&](auto rows2) {
        constexpr int XT = decltype(rows2)::value;
        struct Turn {
            int begin, live;                   // its slots in the list
            bool last;                         // of the item for these slots
            uint32_t d;
            FewWeights<FP4, 1, G> w;
            FewColumns<XT> x;
        };
        // what is loaded next: item, its experts' slots, its turns
        int it = wave - WAVES, count = 0, first = 0, c0 = 0, turn = 0, turn0 = 0, turn1 = 0;
        // (a wave without an item loads through this empty descriptor)
        FewRows<FP4> rows[1] = {FewRows<FP4>(a.w2, a.w2_s, 0, 0, a.I)};
        uint32_t x_off[XT];
        auto set_slots = [&] {
            const int live = count - c0 < kSlots ? count - c0 : kSlots;
#pragma unroll
            for (int j = 0; j < XT; ++j) {
                // SPLIT: row i < 2 is slot i's activations, row 2 + i their remainder
                const int i = SPLIT ? lane >> 5 : 2 * j + (lane >> 5);
                const uint32_t part = SPLIT && j == 1 ? (uint32_t)n * I * 2 : 0u;
                x_off[j] = live > 0 ? (uint32_t)slots[first + c0 + (i < live ? i : 0)] * I * 2 + part : 0u;
            }
            turn = turn0;
        };
        auto next_item = [&] {
            count = c0 = 0;
            for (it += WAVES; it < items; it += WAVES) {           // (experts without slots: none)
                const int ai = it / parts;
                first = __builtin_amdgcn_readfirstlane(begin[ai]);
                count = __builtin_amdgcn_readfirstlane(begin[ai + 1]) - first;
                if (count == 0) continue;
                const int e = __builtin_amdgcn_readfirstlane(expert[ai]), part = it % parts;
                turn0 = part * turns / parts;
                turn1 = (part + 1) * turns / parts;
                rows[0] = FewRows<FP4>(a.w2, a.w2_s, (int64_t)e * a.H + n0, rows_n, a.I);
                break;
            }
            set_slots();
        };
        // the next turn's operands; past the last item no memory is read and there are no slots
        auto load = [&](Turn &q) {
            q.begin = first + c0;
            q.live = count - c0 < kSlots ? count - c0 : kSlots;
            q.d = count ? (uint32_t)turn * kTurn : I;
            q.last = turn + 1 == turn1;
            q.x.lds = lds + at.columns + (size_t)wave * kItemSlots * 512;
            q.x.load(hr, I, q.d, [&](int i) { return x_off[i / 2]; });
            q.w.template load<true>(rows, I, q.d, 0);
            if (++turn == turn1) {
                c0 += kSlots;
                if (c0 < count)
                    set_slots();
                else
                    next_item();
            }
        };
        f32x4 acc[1] = {};
        auto finish = [&](Turn &q) {
            q.x.store();
            q.w.multiply(acc, I, q.d, 0, [&](uint32_t i) { return q.x.chunk(i); }, [&](int i) { return q.w.scales(i); });
            if (!q.last) return;
            if constexpr (SPLIT) {
                // columns c and c + 2 of a quad; an infinite or NaN weight makes
                // the value's sum what it has to be and the remainder's anything
                // (infinity times 0 or the other sign), so that one is left out
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float rest = __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
                        0, (int)__float_as_uint(acc[0][i]), 0x4E, 0xF, 0xF, false));
                    acc[0][i] += __builtin_isfinite(rest) ? rest : 0.0f;
                }
            }
            const bool real = c < q.live;
            const int slot = slots[q.begin + (real ? c : 0)];
            const float wt = wts[slot];
            const int t = slot / a.k;
            // a token that names the expert more than once has those slots side
            // by side: the later ones add in later rounds
            const int prev = __builtin_amdgcn_update_dpp(-1, t, 0x111, 0xF, 0xF, false);       // row_shr:1
            int rank = 0;
            if (__ballot(real && prev == t) != 0) {
                for (int j = 1; j < kSlots; ++j) {
                    const int pt = __shfl(t, (lane & ~15) + (c >= j ? c - j : 0), kWave);
                    if (c >= j && pt == t) ++rank;
                }
            }
            for (int round = 0; __ballot(real && rank >= round) != 0; ++round) {
                if (real && rank == round) {
                    f32x4 *o = reinterpret_cast<f32x4 *>(mine + t * 16 + 4 * g);
                    *o = *o + acc[0] * wt;
                }
            }
            acc[0] = f32x4{};
        };
        auto step = [&](Turn &q) {
            if (q.live <= 0) return false;
            finish(q);
            __builtin_amdgcn_sched_barrier(0);
            load(q);
            __builtin_amdgcn_sched_barrier(0);
            return true;
        };
        next_item();
        Turn q0, q1;
        load(q0);
        load(q1);
        if constexpr (FP4) {
            Turn q2;
            load(q2);
            while (step(q0) && step(q1) && step(q2)) {
            }
        } else {
            while (step(q0) && step(q1)) {
            }
        }
    };
    if constexpr (SPLIT)
        run(std::integral_constant<int, kSplitTokens>{});
    else if (many)
        run(std::integral_constant<int, kItemSlots / 2>{});
    else
        run(std::integral_constant<int, 1>{});
    __syncthreads();
    for (int i = tid; i < a.T * 8; i += WAVES * kWave) {
        const int t = i / 8, j = 2 * (i % 8);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            s0 += sums[((size_t)w * a.T + t) * 16 + j];
            s1 += sums[((size_t)w * a.T + t) * 16 + j + 1];
        }
        if (j < rows_n) *reinterpret_cast<uint32_t *>(a.out + (int64_t)t * a.H + n0 + j) = pack_bf16(s0, s1);
    }
}

}  // namespace

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

namespace {

inline int check_mx_row(int64_t H)
{
    if (H < 1) return CDL_ERR_BAD_SIZE;
    if (H > CDL_MAX_HIDDEN) return CDL_ERR_TOO_LARGE;
    if (H % CDL_MXFP4_GROUP != 0) return CDL_ERR_UNSUPPORTED;
    return CDL_OK;
}

inline unsigned mx_row_blocks(int64_t rows)
{
    const int64_t b = (rows + kMxRowsPerWg - 1) / kMxRowsPerWg;
    return (unsigned)(b < 65536 ? b : 65536);
}

template <bool LL>
int launch_mx_scatter(const uint16_t *x, int64_t T, int64_t H, int32_t k, const int32_t *src2dst, uint8_t *q,
                      uint8_t *s, int64_t cap_rows, int32_t *status, const MxLL &ll, hipStream_t stream)
{
    if (T == 0 && !LL) return CDL_OK;
    const int64_t blocks = T > 0 ? (T + kMxRowsPerWg - 1) / kMxRowsPerWg : 1;
    mx_scatter_kernel<LL><<<dim3((unsigned)blocks), dim3(kMxRowsPerWg * kWave), 0, stream>>>(
        x, T, H, k, src2dst, q, s, cap_rows, status, ll);
    return launch_status();
}

// Small batches (at most 4096 slots) lay themselves out in the launch that
// moves their rows; one token a workgroup up to 512 tokens, 4 above.  Every
// workgroup then counts all slots and scans all experts, so that the layout's
// own kernel and the scatter are the faster where slots, experts and workgroups
// are many (few experts: the counting lanes also meet in the same words).
// Measured, us for the one launch and for the two (H = 512):
//   512 tokens of top-8: 11.1 and 9.2 (8 experts), 11.3 and 13.5 (128), 15.7
//   and 14.5 (1024), 20.0 and 15.7 (2048); top-5, 8 experts: 8.6 and 9.2
//   2048 experts: 128 tokens of top-4 13.6 and 18.9, of top-8 14.8 and 14.2,
//   of top-32 24.0 and 34.8; 512 tokens of top-2 13.7 and 12.3
//   1024 tokens, 32 of 256 experts: top-1 5.2 and 7.8, top-2 6.9 and 7.7,
//   top-4 10.4 and 8.3; 4096 tokens of top-1 19.2 and 10.0
//   1024 tokens of top-2: 128 experts 7.9 and 8.5, 512 experts 9.5 and 8.9
inline bool mx_self_counting(int64_t T, int32_t k, int32_t L)
{
    const int64_t n = T * k;
    if (T > 512) return n + 2 * L <= 2816;
    if (n > 4096) return false;
    if (L > 1024) return n <= 512 || k > 16;
    return (L >= 64 && L <= 512) || T * n <= 3 << 19;
}

template <bool LL>
int launch_mx_permute_self(const PermuteArgs &a, const uint16_t *x, int64_t H, uint8_t *q, uint8_t *s,
                           hipStream_t stream)
{
    const int tpb = a.T <= 512 ? 1 : 4;
    const size_t lds = (size_t)(2 * a.L + tpb * a.k) * sizeof(int32_t);
    const dim3 grid((unsigned)((a.T + tpb - 1) / tpb));
    if (tpb == 1)
        mx_permute_kernel<1, true, LL><<<grid, dim3(2 * kWave), lds, stream>>>(a, x, H, q, s);
    else
        mx_permute_kernel<4, true, LL><<<grid, dim3(5 * kWave), lds, stream>>>(a, x, H, q, s);
    return launch_status();
}

// Longer batches take the layout's own kernels, then the scatter: the layout
// wave of every workgroup adds up the counts of all superblocks, work that
// grows with T and L in each of T / 4 workgroups, and its rows wait for it.
// Wide rows hide more of it.  Measured, us for one launch after the count and
// for the separate layout, top-8, all experts local, T = 2560 / 4096 / 8192:
// H = 2048, L = 128: 19.9 and 24.7 / 30.8 and 27.0 / 62.5 and 39.4;
// H = 7168, L = 128: 27.6 and 34.1 / 46.3 and 47.9 / 108.8 and 101.6;
// H = 16384, 32 of 256 experts: 22.3 and 28.0 / 33.6 and 37.0 / 57.4 and 62.1
// (16384 tokens: top-8 109 and 121, top-2 52 and 47; 32768, top-2: 114 and 83).
// Beyond 3 workgroups a CU (one launch of 704 of them: L = 2048, H = 512, top-8
// 40.8 and 46.9; of 800: 59.5 and 51.3) many experts take the layout apart
// earlier: 800 workgroups of top-8, L = 128: H = 512 24.5 and 22.9, H = 4096
// 31.1 and 31.4; L = 512: H = 2048 36.8 and 35.3, H = 7168 51.2 and 55.8;
// 1024 workgroups of top-8, H = 7168: L = 512 60.1 and 56.8, L = 2048 91.6 and
// 76.9; of top-2, H = 512: L = 32 11.9 and 12.0, L = 2048 45.3 and 32.6.
// Up to 4096 slots the layout is one kernel that counts them itself; those
// batches take it where they do not lay themselves out above.
inline bool mx_layout_apart(int64_t T, int32_t k, int64_t H, int32_t L)
{
    const int64_t blocks = (T + kMaxTpbFp8 - 1) / kMaxTpbFp8;
    if (blocks > 3 * 256 && L > (H <= 2048 ? 32 : H <= 4096 ? 128 : 512)) return true;
    return T * k <= 4096 || T >= (H <= 4096 ? 4096 : H <= kMxPairs * 1024 ? 5121 : 16385);
}

// Batches in between count their superblocks first.
int launch_mx_permute(PermuteArgs a, const uint16_t *x, int64_t H, uint8_t *q, uint8_t *s, void *ws,
                      hipStream_t stream)
{
    const Plan p = make_plan(a.T, a.k, a.L, kMaxTpbFp8);
    a.sb_counts = (const int32_t *)ws;
    a.S = p.S;
    a.sbb_shift = 0;
    while ((int64_t)1 << a.sbb_shift < p.sbb) ++a.sbb_shift;     // sbb is a power of two
    a.sb_slots = p.sb_slots;
    if (p.S * (int64_t)a.L > (int64_t)INT32_MAX) return CDL_ERR_TOO_LARGE;
    layout_count_kernel<<<dim3((unsigned)p.S), dim3(kCountThreads), a.L * sizeof(int32_t), stream>>>(
        a.ids, p.n, p.sb_slots, a.expert_begin, a.L, (int32_t *)ws);
    int rc = launch_status();
    if (rc != CDL_OK) return rc;
    const size_t lds = (size_t)(2 * a.L + p.tpb * a.k) * sizeof(int32_t);
    const dim3 grid((unsigned)p.nblocks);
    switch (p.tpb) {
    case 1: mx_permute_kernel<1, false, false><<<grid, dim3(2 * kWave), lds, stream>>>(a, x, H, q, s); break;
    case 2: mx_permute_kernel<2, false, false><<<grid, dim3(3 * kWave), lds, stream>>>(a, x, H, q, s); break;
    case 4: mx_permute_kernel<4, false, false><<<grid, dim3(5 * kWave), lds, stream>>>(a, x, H, q, s); break;
    default: return CDL_ERR_UNSUPPORTED;       // (8 tokens: only up to 4096 slots, which do not come here)
    }
    return launch_status();
}

int check_grouped(const uint8_t *q, const uint8_t *s, int64_t rows, int64_t K, const uint8_t *wq,
                  const uint8_t *ws, int32_t L, int64_t N, const int32_t *counts, const int64_t *seg, int64_t cap)
{
    if (rows < 0 || K < 1 || N < 1 || L < 1 || L > CDL_MAX_LOCAL_EXPERTS) return CDL_ERR_BAD_SIZE;
    if (!seg && (cap < 0 || rows != (int64_t)L * cap)) return CDL_ERR_BAD_SIZE;
    if (K > CDL_MAX_HIDDEN || N > CDL_MAX_HIDDEN || rows > INT32_MAX) return CDL_ERR_TOO_LARGE;
    if (!counts || !wq || !ws || (rows > 0 && (!q || !s))) return CDL_ERR_NULL_POINTER;
    if (K % CDL_MXFP4_GROUP != 0 || !aligned(q, 16) || !aligned(wq, 16)) return CDL_ERR_UNSUPPORTED;
    return CDL_OK;
}

template <int MT, bool SWIGLU>
int launch_grouped_tiles(const GroupedArgs &a, hipStream_t stream)
{
    constexpr int kCols = SWIGLU ? kGroupedNT / 2 : kGroupedNT;
    const int64_t tiles_n = ((SWIGLU ? a.N / 2 : a.N) + kCols - 1) / kCols;
    // Tiles are numbered in 32 bits, whatever counts the device arrays hold
    // (each is cut to the buffer), with room for a workgroup's step past the
    // last one; every expert adds at most one partly filled row tile.
    const int64_t most = a.seg ? a.rows : a.cap;
    if ((most + MT - 1) / MT * tiles_n > (INT32_MAX - kGroupedWgs) / a.L) return CDL_ERR_TOO_LARGE;
    const int64_t tiles_m = a.seg ? a.rows / MT + a.L : (int64_t)a.L * ((a.cap + MT - 1) / MT);
    const int64_t filled = (tiles_m * tiles_n + 7) / 8 * 8, tiles = filled ? filled : 8;     // (none: the counts' check)
    grouped_kernel<MT, SWIGLU><<<dim3((unsigned)(tiles < kGroupedWgs ? tiles : kGroupedWgs)), dim3(kGroupedThreads),
                                 GroupedShape<MT>::kLds + (size_t)a.L * sizeof(int32_t), stream>>>(a, (int)tiles_n);
    return launch_status();
}

// Tiles of 256 token rows where the buffer has 64 rows or more an expert,
// tiles of 64 below and for padded buffers of up to 256 rows an expert, which
// are mostly empty in decode (the host sees the buffer, not the counts: a larger
// one takes the large tile however empty it is).  Measured, us for tiles of 64 and 256: 4096 rows
// of 32 experts, K = 7168, N = 4096: 165 and 127-133; 9000 rows of 64 uneven
// experts, K = 1440, N = 5000: 137 and 109; 131072 rows of 128 experts,
// K = N = 4096: 2015 and 1269; padded, 128 tokens of top-8 over 32 of 256
// experts, K = 7168, N = 4096: 88 and 93.  At 64 rows an expert drawn at
// random (32 experts, K = 7168, N = 4096) 120 and 108, at 32 rows 93 and 100.
// Tiles of 64 also where they are expected to give every workgroup one at most
// (segments of random length take half a tile more each): 8 experts of 96 rows,
// K = 7168, N = 4096: 38 and 46; of 128 rows, 320 tiles, 65 and 54.
template <bool SWIGLU>
int launch_grouped(const GroupedArgs &a, hipStream_t stream)
{
    // (an empty buffer: only the check of the counts is left)
    if (a.rows == 0 && !a.status) return CDL_OK;
    const int64_t small_tiles = (a.rows / 64 + a.L / 2) * ((a.N + kGroupedNT - 1) / kGroupedNT);
    const bool large = a.seg ? a.rows / a.L >= 64 && small_tiles > kGroupedWgs : a.cap > 256;
    return large ? launch_grouped_tiles<256, SWIGLU>(a, stream) : launch_grouped_tiles<64, SWIGLU>(a, stream);
}

// Tokens whose activations the workspace holds: up to kSplitTokens have the
// remainders as well, and a batch takes no less than a smaller one.
inline int64_t few_act_tokens(int64_t T)
{
    const int64_t split = 2 * (T < kSplitTokens ? T : kSplitTokens);
    return T > split ? T : split;
}

inline int check_few(int64_t T, int32_t k, int64_t H, int64_t I, int32_t L)
{
    int rc = check_tk(T, k);
    if (rc != CDL_OK) return rc;
    if (H < 1 || I < 1 || L < 1 || L > CDL_MAX_LOCAL_EXPERTS) return CDL_ERR_BAD_SIZE;
    if (H > CDL_MAX_HIDDEN || I > CDL_MAX_HIDDEN) return CDL_ERR_TOO_LARGE;
    // the token rows and the activations are addressed with 32-bit byte offsets
    if (T * H > INT32_MAX - 8 || few_act_tokens(T) * k * I > INT32_MAX - 8) return CDL_ERR_TOO_LARGE;
    if (T > CDL_MOE_LAYER_MAX_TOKENS || T * k > kFewMaxSlots) return CDL_ERR_UNSUPPORTED;
    return CDL_OK;
}

inline size_t few_list_bytes(int64_t T, int32_t k, int32_t L)
{
    const int64_t n = T * k;
    return (FewLists::ints(few_experts((int)n, L), n) * sizeof(int32_t) + 255) & ~(size_t)255;
}

inline size_t few_ws_bytes(int64_t T, int32_t k, int64_t I, int32_t L)
{
    return few_list_bytes(T, k, L) + (((size_t)(few_act_tokens(T) * k) * (size_t)I * 2 + 255) & ~(size_t)255);
}

template <bool FP4>
int run_few(FewArgs a, void *ws, hipStream_t stream)
{
    const int n = a.T * a.k;
    a.lists = (int32_t *)ws;
    a.h = (uint16_t *)((uint8_t *)ws + few_list_bytes(a.T, a.k, a.L));
    const int A = few_experts(n, a.L);
    const size_t lists = n > kWave ? ((size_t)n * 2 + 15) / 16 * 16 : 0;
    const dim3 grid1((unsigned)((a.I + 15) / 16), (unsigned)A);
    // scales of 32 rows in LDS (16 KB at H = 16384; one token, H = 7168, I =
    // 2048, top-8: 31 -> 26 us)
    const bool lds_scales = FP4 && a.H <= 16384;
    const size_t lds1 = lists + (lds_scales ? 2 * ((size_t)a.H / 2 + 8) + 64 : 0);
    auto launch = [&](auto xt, auto sc) {
        few_gate_up_kernel<FP4, decltype(xt)::value, decltype(sc)::value><<<grid1, dim3(kFewThreads), lds1, stream>>>(a);
    };
    auto launch_xt = [&](auto sc) {
        if (a.T <= kSplitTokens)
            launch(std::integral_constant<int, kSplitXt>{}, sc);
        else
            launch(std::integral_constant<int, 4>{}, sc);
    };
    if constexpr (FP4) {
        if (lds_scales)
            launch_xt(std::true_type{});
        else
            launch_xt(std::false_type{});
    } else {
        launch_xt(std::false_type{});
    }
    int rc = launch_status();
    if (rc != CDL_OK) return rc;
    const dim3 grid((unsigned)((a.H + 15) / 16));
    // Waves a workgroup: two workgroups a CU where there are that many, by what
    // every wave's sums take of the LDS; otherwise as many as fit.
    static_assert(8 * CDL_MOE_LAYER_MAX_TOKENS * 64 + 8 * kItemSlots * 512 + kFewMaxSlots * 10 + 16 <= 160 * 1024 &&
                      16 * 64 * 64 + 16 * kItemSlots * 512 + 2048 * 10 + 16 <= 160 * 1024,
                  "the second kernel's LDS");
    const bool fill = grid.x < 256;
    auto down = [&](auto waves, auto split) {
        constexpr int W = decltype(waves)::value;
        few_down_kernel<FP4, W, decltype(split)::value><<<grid, dim3(W * kWave), FewDownLds(W, a.T, n, A).bytes, stream>>>(a);
    };
    const std::integral_constant<int, 16> w16;
    const std::integral_constant<int, 8> w8;
    const std::integral_constant<int, 4> w4;
    if (a.T <= kSplitTokens) {
        if (fill)
            down(w16, std::true_type{});
        else
            down(w8, std::true_type{});
    } else if (fill && a.T <= 64 && n <= 2048) {
        down(w16, std::false_type{});
    } else if (fill || a.T <= 64) {
        down(w8, std::false_type{});
    } else {
        down(w4, std::false_type{});
    }
    return launch_status();
}

int moe_layer_call(bool fp4, const uint16_t *x, int64_t T, int64_t H, int32_t k, const int32_t *topk_ids,
                   const float *topk_weights, int32_t expert_begin, int32_t L, int64_t I, const void *w13,
                   const uint8_t *w13_s, const void *w2, const uint8_t *w2_s, uint16_t *out, void *ws,
                   size_t ws_bytes, void *stream)
{
    int rc = check_few(T, k, H, I, L);
    if (rc != CDL_OK) return rc;
    if (T == 0) return CDL_OK;
    if (!x || !topk_ids || !topk_weights || !w13 || !w2 || !out || !ws) return CDL_ERR_NULL_POINTER;
    if (fp4 && (!w13_s || !w2_s)) return CDL_ERR_NULL_POINTER;
    if (ws_bytes < few_ws_bytes(T, k, I, L)) return CDL_ERR_WORKSPACE;
    const int64_t step = fp4 ? CDL_MXFP4_GROUP : 8;
    if (H % step != 0 || I % step != 0) return CDL_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(out, 4) || !aligned(ws, 16))
        return CDL_ERR_UNSUPPORTED;
    FewArgs a = {};
    a.x = x;
    a.ids = topk_ids;
    a.weights = topk_weights;
    a.T = (int32_t)T;
    a.k = k;
    a.expert_begin = expert_begin;
    a.L = L;
    a.H = H;
    a.I = I;
    a.w13 = (const uint8_t *)w13;
    a.w13_s = w13_s;
    a.w2 = (const uint8_t *)w2;
    a.w2_s = w2_s;
    a.out = out;
    return fp4 ? run_few<true>(a, ws, (hipStream_t)stream) : run_few<false>(a, ws, (hipStream_t)stream);
}

}  // namespace

extern "C" {

int cdl_quant_mxfp4(const uint16_t *x, int64_t rows, int64_t H, uint8_t *q, uint8_t *scales, void *stream)
{
    if (rows < 0) return CDL_ERR_BAD_SIZE;
    int rc = check_mx_row(H);
    if (rc != CDL_OK) return rc;
    if (rows == 0) return CDL_OK;
    if (!x || !q || !scales) return CDL_ERR_NULL_POINTER;
    if (!aligned(x, 16) || !aligned(q, 8)) return CDL_ERR_UNSUPPORTED;
    mx_quant_kernel<<<dim3(mx_row_blocks(rows)), dim3(kMxRowsPerWg * kWave), 0, (hipStream_t)stream>>>(x, rows, H, q,
                                                                                                      scales);
    return launch_status();
}

int cdl_dequant_mxfp4(const uint8_t *q, const uint8_t *scales, int64_t rows, int64_t H, uint16_t *out, void *stream)
{
    if (rows < 0) return CDL_ERR_BAD_SIZE;
    int rc = check_mx_row(H);
    if (rc != CDL_OK) return rc;
    if (rows == 0) return CDL_OK;
    if (!q || !scales || !out) return CDL_ERR_NULL_POINTER;
    if (!aligned(q, 8) || !aligned(out, 16)) return CDL_ERR_UNSUPPORTED;
    if (rows > INT64_MAX / 2 / H) return CDL_ERR_TOO_LARGE;
    const int64_t n8 = rows * (H / 8);
    const int64_t blocks = (n8 + 256 * kMxDequantSteps - 1) / (256 * kMxDequantSteps);
    mx_dequant_kernel<<<dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, (hipStream_t)stream>>>(
        (const uint32_t *)q, scales, n8, (u32x4 *)out);
    return launch_status();
}

int cdl_dispatch_mxfp4(const uint16_t *x, int64_t T, int64_t H, int32_t k, const int32_t *src2dst, uint8_t *out_q,
                       uint8_t *out_scales, int64_t cap_rows, int32_t *status, void *stream)
{
    int rc = check_tk(T, k);
    if (rc != CDL_OK) return rc;
    if (cap_rows < 0) return CDL_ERR_BAD_SIZE;
    rc = check_mx_row(H);
    if (rc != CDL_OK) return rc;
    if (cap_rows > INT32_MAX) return CDL_ERR_TOO_LARGE;
    if (T > 0 && (!x || !src2dst)) return CDL_ERR_NULL_POINTER;
    if (cap_rows > 0 && (!out_q || !out_scales)) return CDL_ERR_NULL_POINTER;
    if (!aligned(x, 16) || !aligned(out_q, 8)) return CDL_ERR_UNSUPPORTED;
    return launch_mx_scatter<false>(x, T, H, k, src2dst, out_q, out_scales, cap_rows, status, MxLL{},
                                    (hipStream_t)stream);
}

int cdl_permute_mxfp4(const uint16_t *x, int64_t T, int64_t H, int32_t k, const int32_t *topk_ids,
                      int32_t expert_begin, int32_t L, int32_t alignment, int32_t *counts, int64_t *seg_indptr,
                      int32_t *src2dst, int32_t *reorder_topk_ids, int64_t reorder_cap, uint8_t *out_q,
                      uint8_t *out_scales, int64_t cap_rows, int32_t *status, void *ws, size_t ws_bytes,
                      void *stream)
{
    int rc = check_layout_args(topk_ids, T, k, L, alignment, counts, seg_indptr, src2dst, reorder_topk_ids,
                               reorder_cap, ws, ws_bytes);
    if (rc != CDL_OK) return rc;
    if (cap_rows < 0) return CDL_ERR_BAD_SIZE;
    rc = check_mx_row(H);
    if (rc != CDL_OK) return rc;
    if (cap_rows > INT32_MAX) return CDL_ERR_TOO_LARGE;
    if (T > 0 && !x) return CDL_ERR_NULL_POINTER;
    if (cap_rows > 0 && (!out_q || !out_scales)) return CDL_ERR_NULL_POINTER;
    if (!aligned(x, 16) || !aligned(out_q, 8)) return CDL_ERR_UNSUPPORTED;
    PermuteArgs a = layout_args(topk_ids, T, k, expert_begin, L, alignment, counts, seg_indptr, src2dst,
                                reorder_topk_ids, reorder_cap, status);
    a.cap_rows = cap_rows;
    if (T == 0) return run_layout<kLayoutOnly>(a, ws, (hipStream_t)stream);
    if (mx_self_counting(T, k, L)) return launch_mx_permute_self<false>(a, x, H, out_q, out_scales, (hipStream_t)stream);
    if (mx_layout_apart(T, k, H, L)) {
        rc = run_layout<kLayoutOnly>(a, ws, (hipStream_t)stream);
        if (rc != CDL_OK) return rc;
        return launch_mx_scatter<false>(x, T, H, k, src2dst, out_q, out_scales, cap_rows, status, MxLL{},
                                        (hipStream_t)stream);
    }
    return launch_mx_permute(a, x, H, out_q, out_scales, ws, (hipStream_t)stream);
}

int cdl_permute_ll_mxfp4(const uint16_t *x, int64_t T, int64_t H, int32_t k, const int32_t *topk_ids,
                         int32_t expert_begin, int32_t L, int32_t *counts, int64_t *seg_indptr, int32_t *src2dst,
                         int32_t *reorder_topk_ids, int64_t reorder_cap, int64_t cap, uint8_t *out_q,
                         uint8_t *out_scales, int32_t *masked_m, int32_t *ll_src2dst, int32_t *status, void *ws,
                         size_t ws_bytes, void *stream)
{
    int rc = check_layout_args(topk_ids, T, k, L, 1, counts, seg_indptr, src2dst, reorder_topk_ids, reorder_cap, ws,
                               ws_bytes);
    if (rc != CDL_OK) return rc;
    if (cap < 0) return CDL_ERR_BAD_SIZE;
    rc = check_mx_row(H);
    if (rc != CDL_OK) return rc;
    if (cap > INT32_MAX / L) return CDL_ERR_TOO_LARGE;
    if (!masked_m || (T > 0 && (!x || !ll_src2dst))) return CDL_ERR_NULL_POINTER;
    if (cap > 0 && (!out_q || !out_scales)) return CDL_ERR_NULL_POINTER;
    if (!aligned(x, 16) || !aligned(out_q, 8)) return CDL_ERR_UNSUPPORTED;
    PermuteArgs a = layout_args(topk_ids, T, k, expert_begin, L, 1, counts, seg_indptr, src2dst, reorder_topk_ids,
                                reorder_cap, status);
    if (T > 0 && mx_self_counting(T, k, L)) {
        a.ll_cap = cap;
        a.masked_m = masked_m;
        a.ll_src2dst = ll_src2dst;
        return launch_mx_permute_self<true>(a, x, H, out_q, out_scales, (hipStream_t)stream);
    }
    rc = run_layout<kLayoutOnly>(a, ws, (hipStream_t)stream);
    if (rc != CDL_OK) return rc;
    const MxLL ll = {topk_ids, expert_begin, L, seg_indptr, counts, cap, masked_m, ll_src2dst};
    return launch_mx_scatter<true>(x, T, H, k, src2dst, out_q, out_scales, (int64_t)L * cap, status, ll,
                                   (hipStream_t)stream);
}

int cdl_grouped_mxfp4(const uint8_t *q, const uint8_t *scales, int64_t rows, int64_t K, const uint8_t *w_q,
                      const uint8_t *w_scales, int32_t L, int64_t N, const int32_t *counts,
                      const int64_t *seg_indptr, int64_t cap, uint16_t *out, int32_t *status, void *stream)
{
    int rc = check_grouped(q, scales, rows, K, w_q, w_scales, L, N, counts, seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (rows > 0 && !out) return CDL_ERR_NULL_POINTER;
    GroupedArgs a = {q, scales, rows, K, w_q, w_scales, L, N, counts, seg_indptr, cap, status, out, nullptr, nullptr};
    return launch_grouped<false>(a, (hipStream_t)stream);
}

int cdl_grouped_swiglu_mxfp4(const uint8_t *q, const uint8_t *scales, int64_t rows, int64_t K, const uint8_t *w_q,
                             const uint8_t *w_scales, int32_t L, int64_t I, const int32_t *counts,
                             const int64_t *seg_indptr, int64_t cap, uint8_t *out_q, uint8_t *out_scales,
                             int32_t *status, void *stream)
{
    if (I < 1) return CDL_ERR_BAD_SIZE;
    if (I > CDL_MAX_HIDDEN / 2) return CDL_ERR_TOO_LARGE;
    int rc = check_grouped(q, scales, rows, K, w_q, w_scales, L, 2 * I, counts, seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (rows > 0 && (!out_q || !out_scales)) return CDL_ERR_NULL_POINTER;
    if (I % CDL_MXFP4_GROUP != 0 || !aligned(out_q, 16)) return CDL_ERR_UNSUPPORTED;
    GroupedArgs a = {q, scales, rows, K, w_q, w_scales, L, 2 * I, counts, seg_indptr, cap, status, nullptr, out_q,
                     out_scales};
    return launch_grouped<true>(a, (hipStream_t)stream);
}

size_t cdl_moe_layer_workspace_size(int64_t T, int32_t k, int64_t I, int32_t L)
{
    if (check_few(T, k, 1, I, L) != CDL_OK) return 0;
    return few_ws_bytes(T > 0 ? T : 1, k, I, L);
}

int cdl_moe_layer(const uint16_t *x, int64_t T, int64_t H, int32_t k, const int32_t *topk_ids,
                  const float *topk_weights, int32_t expert_begin, int32_t L, int64_t I, const uint16_t *w13,
                  const uint16_t *w2, uint16_t *out, void *ws, size_t ws_bytes, void *stream)
{
    return moe_layer_call(false, x, T, H, k, topk_ids, topk_weights, expert_begin, L, I, w13, nullptr, w2, nullptr,
                          out, ws, ws_bytes, stream);
}

int cdl_moe_layer_mxfp4(const uint16_t *x, int64_t T, int64_t H, int32_t k, const int32_t *topk_ids,
                        const float *topk_weights, int32_t expert_begin, int32_t L, int64_t I, const uint8_t *w13_q,
                        const uint8_t *w13_scales, const uint8_t *w2_q, const uint8_t *w2_scales, uint16_t *out,
                        void *ws, size_t ws_bytes, void *stream)
{
    return moe_layer_call(true, x, T, H, k, topk_ids, topk_weights, expert_begin, L, I, w13_q, w13_scales, w2_q,
                          w2_scales, out, ws, ws_bytes, stream);
}

}  // extern "C"
