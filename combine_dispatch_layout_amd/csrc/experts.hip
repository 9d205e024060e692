// experts.hip -- MXFP4 rows, the grouped MXFP4 product of the local experts
// and the MoE layer of a few tokens, for MI355X (gfx950).  Included after
// cdl.hip (same translation unit).
//
// MXFP4 (OCP microscaling): groups of 32 elements along a row share a scale
// 2^e, stored as the byte e + 127; an element is an e2m1 code (sign, 2
// exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte,
// the even element in the low half.

namespace {

// ---------------------------------------------------------------------------
// MXFP4 quantisation
// ---------------------------------------------------------------------------

typedef __bf16 v2bf16 __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

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
// code (field 0: 2^-127), and saturates at 6; checked on gfx950 over every
// bf16 for fields 0 to 254.
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

constexpr int kMxPairs = 7;      // blocks of 1024 elements a wave holds: one row at H = 7168

// A wave's row of H elements (from c0 = a multiple of 7 blocks on): loaded,
// quantised and held; lane l of block p has elements 1024 p + 16 l to + 15.
__device__ __forceinline__ void mx_load_row(u32x4 (&v)[2 * kMxPairs], rsrc_t xr, int lane, uint32_t byte0)
{
#pragma unroll
    for (int p = 0; p < kMxPairs; ++p) {
        v[2 * p] = buf_ld16(xr, (uint32_t)lane * 32u + p * 2048u + byte0, 0);
        v[2 * p + 1] = buf_ld16(xr, (uint32_t)lane * 32u + p * 2048u + byte0 + 16u, 0);
    }
}

__device__ __forceinline__ void mx_quant_row(const u32x4 (&v)[2 * kMxPairs], u32x2 (&q)[kMxPairs],
                                             uint32_t (&s)[kMxPairs])
{
#pragma unroll
    for (int p = 0; p < kMxPairs; ++p) q[p] = mx_quant16(v[2 * p], v[2 * p + 1], &s[p]);
}

// The held blocks to destination row dst.  The range check of the row's
// descriptors drops the lanes past the row (H is a multiple of 32: a lane's
// 8 bytes and its group's byte are inside the row or outside as a whole).
__device__ __forceinline__ void mx_store_row(const u32x2 (&q)[kMxPairs], const uint32_t (&s)[kMxPairs],
                                             int lane, uint8_t *oq, uint8_t *os, int64_t dst, int64_t H,
                                             uint32_t block0)
{
    const rsrc_t rq = make_rsrc(oq + dst * (H / 2), (uint32_t)(H / 2));
    const rsrc_t rs = make_rsrc(os + dst * (H / 32), (uint32_t)(H / 32));
#pragma unroll
    for (int p = 0; p < kMxPairs; ++p) {
        if ((int64_t)(block0 + p) * 1024 >= H) break;
        __builtin_amdgcn_raw_buffer_store_b64(q[p], rq, (uint32_t)lane * 8u + (block0 + p) * 512u, 0, 0);
        if ((lane & 1) == 0)
            __builtin_amdgcn_raw_buffer_store_b8((uint8_t)s[p], rs, (uint32_t)lane / 2 + (block0 + p) * 32u, 0, 0);
    }
}

constexpr int kMxRowsPerWg = 4;      // rows (waves) per workgroup

// Rows quantised in place order: out row r from x row r.
__global__ __launch_bounds__(kMxRowsPerWg *kWave) void mx_quant_kernel(
    const uint16_t *__restrict__ x, int64_t rows, int64_t H, uint8_t *__restrict__ q, uint8_t *__restrict__ s)
{
    const int lane = threadIdx.x & (kWave - 1);
    for (int64_t r = (int64_t)blockIdx.x * kMxRowsPerWg + wave_id(); r < rows;
         r += (int64_t)gridDim.x * kMxRowsPerWg) {
        const rsrc_t xr = make_rsrc(x + r * H, (uint32_t)(H * 2));
        for (uint32_t b0 = 0; (int64_t)b0 * 1024 < H; b0 += kMxPairs) {
            u32x4 v[2 * kMxPairs];
            u32x2 c[kMxPairs];
            uint32_t sc[kMxPairs];
            mx_load_row(v, xr, lane, b0 * 2048u);
            mx_quant_row(v, c, sc);
            mx_store_row(c, sc, lane, q, s, r, H, b0);
        }
    }
}

// Codes back to bf16 (exact: three significant bits, exponents in bf16's
// range; 6 * 2^127 and 4 * 2^126 overflow to infinity).  16 elements a thread.
__global__ __launch_bounds__(256) void mx_dequant_kernel(const u32x2 *__restrict__ q, const uint8_t *__restrict__ s,
                                                         int64_t n16, u32x4 *__restrict__ out)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += (int64_t)gridDim.x * 256) {
        const u32x2 c = q[i];
        const float p = __uint_as_float((uint32_t)s[i >> 1] << 23);
        uint32_t o[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = h ? c.y : c.x;
            o[4 * h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 0));
            o[4 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 1));
            o[4 * h + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 2));
            o[4 * h + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 3));
        }
        out[2 * i] = u32x4{o[0], o[1], o[2], o[3]};
        out[2 * i + 1] = u32x4{o[4], o[5], o[6], o[7]};
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
    const uint64_t dmask = __ballot(d >= 0);
    if (dmask == 0) return;
    const rsrc_t xr = make_rsrc(x + t * H, (uint32_t)(H * 2));
    for (uint32_t b0 = 0; (int64_t)b0 * 1024 < H; b0 += kMxPairs) {
        u32x4 v[2 * kMxPairs];
        u32x2 c[kMxPairs];
        uint32_t sc[kMxPairs];
        mx_load_row(v, xr, lane, b0 * 2048u);
        mx_quant_row(v, c, sc);
        for (uint64_t m = dmask; m; m &= m - 1) {
            const int32_t dst = __builtin_amdgcn_readlane(d, (int)__builtin_ctzll(m));
            mx_store_row(c, sc, lane, oq, os, dst, H, b0);
        }
    }
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

// The tile of workgroup `blk`: tiles are ordered by expert, then column tile,
// then row tile (the row tiles of one weight tile run side by side, so its
// second reader finds it in a cache), and each XCD (workgroup index mod 8)
// takes one contiguous eighth of them.  Every wave does this by itself, 64
// experts at a time.  false: no tile.
template <int MT>
__device__ __forceinline__ bool grouped_tile(const GroupedArgs &a, int tiles_n, uint32_t blk, GroupedTile *t)
{
    const int lane = threadIdx.x & (kWave - 1);
    int32_t total = 0;
    bool any_bad = false;
    for (int e0 = 0; e0 < a.L; e0 += kWave) {
        int32_t c = 0;
        if (e0 + lane < a.L) {
            int64_t b;
            bool bad;
            c = (int32_t)((grouped_rows(a, e0 + lane, &b, &bad) + MT - 1) / MT) * tiles_n;
            any_bad |= bad;
        }
        total += __builtin_amdgcn_readlane(wave_inclusive_scan(c), kWave - 1);
    }
    if (blk == 0 && __ballot(any_bad) != 0 && threadIdx.x == 0)
        set_status(a.status, a.seg ? CDL_STATUS_ROWS_OVERFLOW : CDL_STATUS_LL_OVERFLOW);
    const uint32_t per = ((uint32_t)total + 7) / 8;
    const uint32_t id = (blk & 7) * per + (blk >> 3);
    if ((blk >> 3) >= per || id >= (uint32_t)total) return false;
    int32_t base = 0;
    for (int e0 = 0; e0 < a.L; e0 += kWave) {
        int32_t c = 0;
        int64_t b = 0, cnt = 0;
        if (e0 + lane < a.L) {
            bool bad;
            cnt = grouped_rows(a, e0 + lane, &b, &bad);
            c = (int32_t)((cnt + MT - 1) / MT) * tiles_n;
        }
        const int32_t incl = base + wave_inclusive_scan(c);
        const uint64_t hit = __ballot((int32_t)id >= incl - c && (int32_t)id < incl);
        if (hit) {
            const int l = (int)__builtin_ctzll(hit);
            const int32_t mt = __builtin_amdgcn_readlane(c, l) / tiles_n;
            const int32_t local = (int32_t)id - (__builtin_amdgcn_readlane(incl, l) - mt * tiles_n);
            t->e = e0 + l;
            t->n = local / mt;
            t->m = local % mt;
            t->begin = ((int64_t)__builtin_amdgcn_readlane((int)(b >> 32), l) << 32) |
                       (uint32_t)__builtin_amdgcn_readlane((int)b, l);
            t->count = (uint32_t)__builtin_amdgcn_readlane((int)cnt, l);
            return true;
        }
        base = __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    return false;
}

__device__ __forceinline__ i32x8 mx_frag(u32x4 v)
{
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// 32 SwiGLU values of one row across a lane and its partner (lane ^ 32): the
// lane holds values 8 b + 4 (lane / 32) + i at h[4 b + i].  Stores the 16
// code bytes and the scale byte of the group.
__device__ __forceinline__ void store_swiglu_group(const float (&h)[16], int lane, bool live, uint8_t *q, uint8_t *s)
{
    float am = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        am = fmaxf(am, fabsf(h[i]));
        nan |= h[i] != h[i];
    }
    am = fmaxf(am, __shfl_xor(am, 32, kWave));
    nan |= (bool)__shfl_xor((int)nan, 32, kWave);
    // smallest b >= 0 with 6 * 2^(b - 127) >= am, as mx_scale_byte, on the fp32 bits
    const uint32_t bits = __float_as_uint(am);
    const int E = (int)(bits >> 23);
    int b = E - 2 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
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
    // upper: 4-7, 12-15 | 20-23, 28-31.  The lower lane takes the first 8
    // bytes, the upper the last 8.
    const uint32_t o0 = __shfl_xor(c[0], 32, kWave), o1 = __shfl_xor(c[1], 32, kWave);
    const bool up = lane >= 32;
    const uint32_t lo = up ? o1 : c[0], hi = up ? c[1] : o0;
    if (!live) return;
    const u32x2 w = {(lo & 0xFFFFu) | (hi << 16), (lo >> 16) | (hi & 0xFFFF0000u)};
    *reinterpret_cast<u32x2 *>(q + (up ? 8 : 0)) = w;
    if (!up) *s = nan ? (uint8_t)255 : (uint8_t)b;
}

// One wave per tile of 32 weight rows (SwiGLU: 32 gate and 32 up rows) and 32
// token rows, operands straight from memory.  v_mfma_scale_f32_32x32x64: lane
// l holds row l % 32 of its operand and the 32 elements of group l / 32 (16
// bytes, one scale byte); D has token column l % 32 and, in register i,
// weight row 8 (i / 4) + 4 (l / 32) + i % 4.
template <bool SWIGLU>
__global__ __launch_bounds__(kWave) void grouped_kernel(GroupedArgs a, int tiles_n)
{
    GroupedTile t;
    if (!grouped_tile<32>(a, tiles_n, blockIdx.x, &t)) return;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t K2 = a.K / 2, K32 = a.K / 32;
    const int64_t m0 = (int64_t)t.m * 32, n0 = (int64_t)t.n * 32;
    const int64_t I = a.N / 2;
    const int64_t live_m = t.count - m0 < 32 ? t.count - m0 : 32;
    const int64_t n_rows = SWIGLU ? I : a.N;
    const int64_t live_n = n_rows - n0 < 32 ? n_rows - n0 : 32;
    const int r = lane & 31, g = lane >> 5;
    const rsrc_t rq = make_rsrc(a.q + (t.begin + m0) * K2, (uint32_t)(live_m * K2));
    const rsrc_t rs = make_rsrc(a.s + (t.begin + m0) * K32, (uint32_t)(live_m * K32));
    constexpr int NW = SWIGLU ? 2 : 1;
    rsrc_t wq[NW], ws[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const int64_t row = (int64_t)t.e * a.N + i * I + n0;
        wq[i] = make_rsrc(a.wq + row * K2, (uint32_t)(live_n * K2));
        ws[i] = make_rsrc(a.ws + row * K32, (uint32_t)(live_n * K32));
    }
    f32x16 acc[NW] = {};
    for (int64_t g0 = 0; g0 < K32; g0 += 2) {
        // a group past the row's end (odd K / 32) reads an address out of range: zeros
        const bool in = g0 + g < K32;
        const uint32_t vo = in ? (uint32_t)(r * K2 + (g0 + g) * 16) : 0xFFFFFFF0u;
        const uint32_t so = in ? (uint32_t)(r * K32 + g0 + g) : 0xFFFFFFF0u;
        const u32x4 b = buf_ld16(rq, vo, 0);
        const int sb = (int)__builtin_amdgcn_raw_buffer_load_b8(rs, so, 0, 0);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const u32x4 w = buf_ld16(wq[i], vo, 0);
            const int sw = (int)__builtin_amdgcn_raw_buffer_load_b8(ws[i], so, 0, 0);
            acc[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_frag(w), mx_frag(b), acc[i], 4, 4, 0, sw, 0, sb);
        }
    }
    const bool live = r < live_m;
    const int64_t row = t.begin + m0 + r;
    if constexpr (SWIGLU) {
        float h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = acc[0][i] / (1.0f + __expf(-acc[0][i])) * acc[1][i];
        store_swiglu_group(h, lane, live, a.hq + row * (I / 2) + n0 / 2, a.hs + row * (I / 32) + n0 / 32);
    } else {
        if (!live) return;
        uint16_t *o = a.out + row * a.N + n0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int n = 8 * (i / 4) + 4 * g + i % 4;
            if (n < live_n) o[n] = (uint16_t)(pack_bf16_rne(acc[0][i], 0.0f) & 0xFFFFu);
        }
    }
}

// ---------------------------------------------------------------------------
// the MoE layer of a few tokens
// ---------------------------------------------------------------------------

constexpr int kFewThreads = 256;        // first kernel: 4 waves share the columns, split the depth
constexpr int kFewWaves2 = 8;           // second kernel
constexpr int kFewChunk = 512;          // depth of one item of the second kernel
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
    uint16_t *h;                 // [T k, I]
};

// Routing lists in the workspace, written by the first kernel's workgroup 0:
// the number of experts with slots, then for the a-th of them its index and
// the begin of its slots, then the slots (flat t * k + j, ascending).
struct FewLists {
    int32_t *active, *expert, *begin, *slots;
    __host__ __device__ FewLists(int32_t *p, int A) : active(p), expert(p + 4), begin(p + 4 + A), slots(p + 4 + 2 * A + 4) {}
    static size_t ints(int64_t A, int64_t n) { return (size_t)(4 + A + A + 4 + n); }
};

// A 16-row operand fragment of v_mfma_f32_16x16x32_bf16 for one step: lane l
// holds row l % 16 and 8 consecutive elements.  MXFP4 weights: a lane's 16
// bytes are one group of 32 elements, which serve 4 steps of 8.
template <bool FP4>
struct FewStep {
    static constexpr int kDepth = FP4 ? 128 : 32;         // elements of the contraction per load
    static constexpr int kSteps = FP4 ? 4 : 1;            // matrix instructions per load
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

// acc[i] += W_i (16 rows each) * B over the depth steps [d0, d1) with stride:
// W_i rows and the lane's B row (bf16, 16 columns) through descriptors, which
// return zeros past a row block's or row's end.
//   wq[i], ws[i]  descriptors of the 16 weight rows (scales: FP4 only)
//   br            descriptor of the lane's operand rows' common base, b_off the lane's row offset in bytes
template <bool FP4, int NW>
__device__ __forceinline__ void few_product(f32x4 (&acc)[NW], const rsrc_t (&wq)[NW], const rsrc_t (&ws)[NW],
                                            const uint16_t *brow, int64_t depth, int64_t d0, int64_t d1,
                                            int64_t stride)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int r = lane & 15, g = lane >> 4;
    for (int64_t d = d0; d < d1; d += stride) {
        if constexpr (FP4) {
            const int64_t at = d + 32 * g;
            const bool in = at < depth;
            const uint32_t wo = in ? (uint32_t)(r * (depth / 2) + at / 2) : 0xFFFFFFF0u;
            const uint32_t so = in ? (uint32_t)(r * (depth / 32) + at / 32) : 0xFFFFFFF0u;
            u32x4 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = in ? *reinterpret_cast<const u32x4 *>(brow + at + 8 * i) : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const u32x4 w = buf_ld16(wq[i], wo, 0);
                const float p = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b8(ws[i], so, 0, 0) << 23);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_expand<0>(w, p), __builtin_bit_cast(v8bf16, b[0]), acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_expand<1>(w, p), __builtin_bit_cast(v8bf16, b[1]), acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_expand<2>(w, p), __builtin_bit_cast(v8bf16, b[2]), acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(few_expand<3>(w, p), __builtin_bit_cast(v8bf16, b[3]), acc[i], 0, 0, 0);
            }
        } else {
            const int64_t at = d + 8 * g;
            const bool in = at < depth;
            const uint32_t wo = in ? (uint32_t)(r * (depth * 2) + at * 2) : 0xFFFFFFF0u;
            const u32x4 b = in ? *reinterpret_cast<const u32x4 *>(brow + at) : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const u32x4 w = buf_ld16(wq[i], wo, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf16, w), __builtin_bit_cast(v8bf16, b), acc[i], 0, 0, 0);
            }
        }
    }
}

template <bool FP4>
__device__ __forceinline__ void few_weight_rows(const uint8_t *w, const uint8_t *s, int64_t row, int64_t rows,
                                                int64_t depth, rsrc_t *q, rsrc_t *sc)
{
    if constexpr (FP4) {
        *q = make_rsrc(w + row * (depth / 2), (uint32_t)(rows * (depth / 2)));
        *sc = make_rsrc(s + row * (depth / 32), (uint32_t)(rows * (depth / 32)));
    } else {
        *q = make_rsrc(w + row * depth * 2, (uint32_t)(rows * depth * 2));
        *sc = *q;
    }
}

// First kernel: h[slot, i] = silu(gate) * up for 16 columns i of the a-th
// active expert (blockIdx.y); blockIdx.x the column tile.
template <bool FP4>
__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(FewArgs a)
{
    extern __shared__ int32_t lds[];
    int32_t *hist = lds;                       // [L]
    int32_t *list = lds + a.L;                 // [n] the expert's slots
    int16_t *es = reinterpret_cast<int16_t *>(list + a.T * a.k);   // [n] local expert of each slot
    __shared__ f32x4 part[4][2][kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    const int n = a.T * a.k;
    for (int e = tid; e < a.L; e += kFewThreads) hist[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kFewThreads) {
        const int e = local_expert(a.ids[i], a.expert_begin, a.L);
        es[i] = (int16_t)e;
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    // the blockIdx.y-th expert with slots, and the slots of those before it
    int mine = -1, seen = 0, before = 0;
    int32_t slots_seen = 0;
    for (int e0 = 0; e0 < a.L; e0 += kWave) {
        const int32_t c = e0 + lane < a.L ? hist[e0 + lane] : 0;
        const uint64_t m = __ballot(c > 0);
        const int rank = seen + __popcll(m & (lane ? ~0ull >> (kWave - lane) : 0ull));
        const int32_t incl = slots_seen + wave_inclusive_scan(c);
        const uint64_t hit = __ballot(c > 0 && rank == (int)blockIdx.y);
        if (hit) {
            const int l = (int)__builtin_ctzll(hit);
            mine = e0 + l;
            before = __builtin_amdgcn_readlane(incl - c, l);
        }
        seen += __popcll(m);
        slots_seen = __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    // the routing lists of the second kernel: every expert's first workgroup
    // writes the expert's own
    const FewLists ls(a.lists, n < a.L ? n : a.L);
    const bool publish = blockIdx.x == 0 && wave == 0;
    if (publish && lane == 0) {
        if (blockIdx.y == 0) ls.active[0] = seen;
        if (mine >= 0) {
            ls.expert[blockIdx.y] = mine;
            ls.begin[blockIdx.y] = before;
            ls.begin[blockIdx.y + 1] = before + hist[mine];
        }
    }
    if (mine < 0) return;
    if (wave == 0) {
        int at = 0;
        for (int i0 = 0; i0 < n; i0 += kWave) {
            const bool is = i0 + lane < n && es[i0 + lane] == mine;
            const uint64_t m = __ballot(is);
            if (is) {
                const int to = at + __popcll(m & (lane ? ~0ull >> (kWave - lane) : 0ull));
                list[to] = i0 + lane;
                if (publish) ls.slots[before + to] = i0 + lane;
            }
            at += __popcll(m);
        }
    }
    const int count = hist[mine];
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * 16;
    const int64_t rows = a.I - i0 < 16 ? a.I - i0 : 16;
    rsrc_t wq[2], ws[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        few_weight_rows<FP4>(a.w13, a.w13_s, (int64_t)mine * 2 * a.I + i * a.I + i0, rows, a.H, &wq[i], &ws[i]);
    const int c = lane & 15, g = lane >> 4;
    for (int c0 = 0; c0 < count; c0 += 16) {
        const int slot = list[c0 + c < count ? c0 + c : c0];
        const uint16_t *xrow = a.x + (int64_t)(slot / a.k) * a.H;
        f32x4 acc[2] = {};
        constexpr int D = FewStep<FP4>::kDepth;
        few_product<FP4, 2>(acc, wq, ws, xrow, a.H, (int64_t)wave * D, a.H, 4 * D);
        if (c0) __syncthreads();               // the sums of the round before are read
        part[wave][0][lane] = acc[0];
        part[wave][1][lane] = acc[1];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int w = 1; w < 4; ++w) {
                acc[0] += part[w][0][lane];
                acc[1] += part[w][1][lane];
            }
            if (c0 + c < count) {
                float h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = acc[0][i] / (1.0f + __expf(-acc[0][i])) * acc[1][i];
                if (4 * g < rows)
                    *reinterpret_cast<u32x2 *>(a.h + (int64_t)slot * a.I + i0 + 4 * g) =
                        u32x2{pack_bf16_rne(h[0], h[1]), pack_bf16_rne(h[2], h[3])};
            }
        }
    }
}

// Second kernel: out[t, n] for 16 columns n and every token.  The items
// (expert, depth chunk) are dealt to the waves; each wave adds its weighted
// products into sums of its own in LDS, which are added in wave order.
template <bool FP4>
__global__ __launch_bounds__(kFewWaves2 *kWave) void few_down_kernel(FewArgs a)
{
    extern __shared__ float sums[];            // [waves][T][16]
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = wave_id();
    const int n = a.T * a.k;
    const FewLists ls(a.lists, n < a.L ? n : a.L);
    float *mine = sums + (size_t)wave * a.T * 16;
    for (int i = lane; i < a.T * 16; i += kWave) mine[i] = 0.0f;
    const int active = ls.active[0];
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t rows = a.H - n0 < 16 ? a.H - n0 : 16;
    const int chunks = (int)((a.I + kFewChunk - 1) / kFewChunk);
    const int c = lane & 15, g = lane >> 4;
    for (int it = wave; it < active * chunks; it += kFewWaves2) {
        const int ai = it / chunks;
        const int64_t d0 = (int64_t)(it % chunks) * kFewChunk;
        const int64_t d1 = d0 + kFewChunk < a.I ? d0 + kFewChunk : a.I;
        const int e = ls.expert[ai];
        const int begin = ls.begin[ai], count = ls.begin[ai + 1] - begin;
        rsrc_t wq[1], ws[1];
        few_weight_rows<FP4>(a.w2, a.w2_s, (int64_t)e * a.H + n0, rows, a.I, &wq[0], &ws[0]);
        for (int c0 = 0; c0 < count; c0 += 16) {
            const bool real = c0 + c < count;
            const int slot = ls.slots[begin + (real ? c0 + c : c0)];
            f32x4 acc[1] = {};
            few_product<FP4, 1>(acc, wq, ws, a.h + (int64_t)slot * a.I, a.I, d0, d1, FewStep<FP4>::kDepth);
            const float wt = real ? a.weights[slot] : 0.0f;
            const int t = slot / a.k;
            // a token that names the expert twice has both slots side by
            // side: the later ones add in a later round
            int rank = 0;
            for (int j = 1; j < 16; ++j) {
                const int pt = __shfl(t, (lane & ~15) + (c >= j ? c - j : 0), kWave);
                if (c >= j && pt == t) ++rank;
            }
            for (int round = 0; __ballot(real && rank >= round) != 0; ++round) {
                if (real && rank == round) {
                    f32x4 *o = reinterpret_cast<f32x4 *>(mine + t * 16 + 4 * g);
                    *o = *o + acc[0] * wt;
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * 8; i += kFewWaves2 * kWave) {
        const int t = i / 8, j = 2 * (i % 8);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWaves2; ++w) {
            s0 += sums[((size_t)w * a.T + t) * 16 + j];
            s1 += sums[((size_t)w * a.T + t) * 16 + j + 1];
        }
        if (j < rows) *reinterpret_cast<uint32_t *>(a.out + (int64_t)t * a.H + n0 + j) = pack_bf16_rne(s0, s1);
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

template <bool SWIGLU>
int launch_grouped(const GroupedArgs &a, hipStream_t stream)
{
    if (a.rows == 0) return CDL_OK;
    constexpr int MT = 32, NT = 32;
    const int64_t tiles_n = ((SWIGLU ? a.N / 2 : a.N) + NT - 1) / NT;
    // every expert adds at most one partly filled row tile
    const int64_t tiles_m = a.seg ? a.rows / MT + a.L : (int64_t)a.L * ((a.cap + MT - 1) / MT);
    const int64_t grid = (tiles_m * tiles_n + 7) / 8 * 8;
    if (grid > INT32_MAX) return CDL_ERR_TOO_LARGE;
    grouped_kernel<SWIGLU><<<dim3((unsigned)grid), dim3(kWave), 0, stream>>>(a, (int)tiles_n);
    return launch_status();
}

inline int check_few(int64_t T, int32_t k, int64_t H, int64_t I, int32_t L)
{
    int rc = check_tk(T, k);
    if (rc != CDL_OK) return rc;
    if (H < 1 || I < 1 || L < 1 || L > CDL_MAX_LOCAL_EXPERTS) return CDL_ERR_BAD_SIZE;
    if (H > CDL_MAX_HIDDEN || I > CDL_MAX_HIDDEN) return CDL_ERR_TOO_LARGE;
    if (T > CDL_MOE_LAYER_MAX_TOKENS || T * k > kFewMaxSlots) return CDL_ERR_UNSUPPORTED;
    return CDL_OK;
}

inline size_t few_list_bytes(int64_t T, int32_t k, int32_t L)
{
    const int64_t n = T * k;
    return (FewLists::ints(n < L ? n : L, n) * sizeof(int32_t) + 255) & ~(size_t)255;
}

inline size_t few_ws_bytes(int64_t T, int32_t k, int64_t I, int32_t L)
{
    return few_list_bytes(T, k, L) + (((size_t)(T * k) * (size_t)I * 2 + 255) & ~(size_t)255);
}

template <bool FP4>
int run_few(FewArgs a, void *ws, hipStream_t stream)
{
    const int n = a.T * a.k;
    a.lists = (int32_t *)ws;
    a.h = (uint16_t *)((uint8_t *)ws + few_list_bytes(a.T, a.k, a.L));
    const size_t lds1 = (size_t)a.L * 4 + (size_t)n * 4 + (size_t)n * 2;
    few_gate_up_kernel<FP4><<<dim3((unsigned)((a.I + 15) / 16), (unsigned)(n < a.L ? n : a.L)), dim3(kFewThreads),
                              lds1, stream>>>(a);
    int rc = launch_status();
    if (rc != CDL_OK) return rc;
    few_down_kernel<FP4><<<dim3((unsigned)((a.H + 15) / 16)), dim3(kFewWaves2 * kWave),
                           (size_t)kFewWaves2 * a.T * 64, stream>>>(a);
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
    const int64_t n16 = rows * (H / 16);
    const int64_t blocks = (n16 + 255) / 256;
    mx_dequant_kernel<<<dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, (hipStream_t)stream>>>(
        (const u32x2 *)q, scales, n16, (u32x4 *)out);
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
    rc = run_layout<kLayoutOnly>(a, ws, (hipStream_t)stream);
    if (rc != CDL_OK) return rc;
    return launch_mx_scatter<false>(x, T, H, k, src2dst, out_q, out_scales, cap_rows, status, MxLL{},
                                    (hipStream_t)stream);
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
