// norm.hip -- the root-mean-square norm of token rows with the residual's
// addition, as bf16 rows or quantised to fp8, its gradient, and the fp8
// conversions outside a scatter, for MI355X (gfx950).  Included after
// products.hip (same translation unit).

namespace {

// ---------------------------------------------------------------------------
// y = h * r * w with r = 1 / sqrt(mean(h^2) + eps), h = bf16(x + residual)
//
// A row is read once and stays in registers: a workgroup of 256 threads (one
// wave for up to 1024 columns) holds up to 32 elements of it a thread, units of
// 8 (16 bytes) or, where rows are not 16-byte aligned, of 1.  Longer rows are
// read twice.  Bound by the rows' bytes: 4096 x 7168 with residual to fp8 39 to
// 41 us (206 MB, 5.1 TB/s), with the bf16 rows as well 45 (264 MB, 5.9), 16384 x
// 4096 to bf16 83 to 94 us (537 MB, 5.7 to 6.4 TB/s).  Rows of units of 1 take
// about three times as long: 4096 x 7167 122 us against 37.
// ---------------------------------------------------------------------------
constexpr int kNormThreads = 256;
constexpr int kNormHeld = 32 * kNormThreads;     // columns of a row held in registers

struct NormArgs {
    const uint16_t *x, *res, *w;
    float eps;
    int64_t T, H;
    uint16_t *out, *res_out;
    uint8_t *q;                  // fp8: [T, H] and the scales
    void *s;
    int32_t flags;
    ScaleWords words;
};

// VEC bf16 of memory, raw.
template <int VEC>
struct Unit {
    uint32_t v[VEC == 8 ? 4 : 1];
    __device__ __forceinline__ void load(const uint16_t *p)
    {
        if constexpr (VEC == 8) {
            const u32x4 u = *reinterpret_cast<const u32x4 *>(p);
            v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
        } else {
            v[0] = *p;
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (auto &u : v) u = 0;
    }
    __device__ __forceinline__ float at(int i) const
    {
        return VEC == 8 && (i & 1) ? bf16_hi(v[i / 2]) : __uint_as_float(v[VEC == 8 ? i / 2 : 0] << 16);
    }
    __device__ __forceinline__ void store(uint16_t *p) const
    {
        if constexpr (VEC == 8)
            *reinterpret_cast<u32x4 *>(p) = u32x4{v[0], v[1], v[2], v[3]};
        else
            *p = (uint16_t)v[0];
    }
    __device__ __forceinline__ void set(const float (&f)[VEC])
    {
        if constexpr (VEC == 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        } else {
            v[0] = pack_bf16(f[0], 0.0f) & 0xFFFFu;
        }
    }
    // this + o, rounded to bf16.  The fp32 sum rounds to the same bf16 as the
    // exact one: it is itself inexact only where the exponents are more than 16
    // apart, too far for the smaller value to reach a rounding border.
    __device__ __forceinline__ void add(const Unit &o)
    {
        float f[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = at(i) + o.at(i);
        set(f);
    }
};

// Sum of every lane's value, in all lanes.
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int x = 1; x < kWave; x *= 2) v += __shfl_xor(v, x);
    return v;
}

// Sums over a row's threads: a wave, or the workgroup's four, in 64 bits, whose
// additions cost nothing beside the row's loads: the last ones of a tree carry
// most of its rounding.
template <int N, bool WAVE>
__device__ __forceinline__ void row_sums(const double (&v)[N], double (&s)[N], double *lds)
{
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = wave_sum(v[i]);
    if constexpr (!WAVE) {
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) lds[wave * N + i] = s[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = (lds[i] + lds[N + i]) + (lds[2 * N + i] + lds[3 * N + i]);
        __syncthreads();
    }
}

// s + the squares of a unit, in 64 bits (a conversion and an addition an
// element, hidden behind the row's loads: 4096 x 7168 to fp8 39 us either way):
// an error of r moves values of a whole row across fp8's borders, and a sum in 32
// bits loses small squares beside large ones, and the range of rows beyond 2^64.
template <int VEC>
__device__ __forceinline__ double add_squares(const Unit<VEC> &h, double s)
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) s = fma((double)h.at(i), (double)h.at(i), s);
    return s;
}

// 1 / sqrt(sum / H + eps)
__device__ __forceinline__ double row_scale(double sum, int64_t H, float eps)
{
    return 1.0 / sqrt(sum / (double)H + (double)eps);
}

// A row's scale r = 2^e (hi + lo), hi of 1 to 2.  h 2^e is exact and at most
// sqrt(H) in size, and its product with w too, so that y = h w r is rounded once
// (as few values as can be land on the other side of a border of fp8) and nothing
// before it leaves fp32's range.  The correction is held finite: beside an
// infinite product it may be infinite the other way, or NaN.
struct RowScale {
    float power, hi, lo;
    __device__ __forceinline__ explicit RowScale(double r)
    {
        // (the exponent by bit operations: 4096 x 7168 to fp8 41.8 against 39.3 us)
        int e = ilogb(r);                                    // (extreme for a row of zeros or with an infinity)
        e = e < -126 ? -126 : e > 127 ? 127 : e;
        power = ldexpf(1.0f, e);
        r = ldexp(r, -e);
        hi = (float)r;
        lo = (float)(r - (double)hi);
    }
    __device__ __forceinline__ float times(float h, float w) const
    {
        const float v = h * power * w;
        return fmaf(v, hi, __builtin_amdgcn_fmed3f(v * lo, -__FLT_MAX__, __FLT_MAX__));
    }
};

// The scale of group g of row t (lanes of a group share it; lane 16 j of the
// wave stores, or lane 0 a word of four groups, which begin at a multiple of
// four: `first` is the wave's first group).
__device__ __forceinline__ void store_scale(const NormArgs &a, const Fp8Group &q, int64_t t, int64_t g, int64_t first, bool live)
{
    const int lane = threadIdx.x & (kWave - 1);
    if (a.flags & CDL_FP8_SCALE_PACKED) {
        const uint32_t b = live ? q.exponent() : 0u;
        const uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)b, 0) | (uint32_t)__builtin_amdgcn_readlane((int)b, 16) << 8 |
                           (uint32_t)__builtin_amdgcn_readlane((int)b, 32) << 16 | (uint32_t)__builtin_amdgcn_readlane((int)b, 48) << 24;
        if (lane == 0 && live) static_cast<uint32_t *>(a.s)[t * a.words.row + first / 4 * a.words.batch] = w;
    } else if ((lane & 15) == 0 && live) {
        static_cast<float *>(a.s)[t * a.words.row + g * (a.words.group ? a.words.group : 1)] = q.scale;
    }
}

// 8 values of a row's group (16 lanes) to codes.
__device__ __forceinline__ u32x2 quant8(const float (&y)[8], const Fp8Group &q)
{
    uint32_t c[2];
    q.codes<2>(y, c);
    return u32x2{c[0], c[1]};
}

template <int VEC, int NU, bool WAVE, bool FP8>
__global__ __launch_bounds__(kNormThreads) void rms_norm_kernel(NormArgs a)
{
    constexpr int P = WAVE ? kWave : kNormThreads;           // threads of a row
    __shared__ double lds[4];
    const int tid = threadIdx.x % P;
    constexpr int kRows = kNormThreads / P;                  // rows of a workgroup
    const int64_t H = a.H;
    // (t is the same for a wave, and without WAVE for the workgroup)
    for (int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / P; t < a.T; t += (int64_t)gridDim.x * kRows) {
        const int64_t row = t * H;
        Unit<VEC> h[NU], w[NU];
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const int64_t c = (int64_t)(tid + j * P) * VEC;
            h[j].clear();
            w[j].clear();
            if (c < H) h[j].load(a.x + row + c);
        }
        if (a.res) {
            Unit<VEC> r[NU];
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int64_t c = (int64_t)(tid + j * P) * VEC;
                r[j].clear();
                if (c < H) r[j].load(a.res + row + c);
            }
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int64_t c = (int64_t)(tid + j * P) * VEC;
                h[j].add(r[j]);
                if (c < H) h[j].store(a.res_out + row + c);
            }
        }
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const int64_t c = (int64_t)(tid + j * P) * VEC;
            if (c < H) w[j].load(a.w + c);
        }
        double sum[1] = {0.0};
#pragma unroll
        for (int j = 0; j < NU; ++j) sum[0] = add_squares(h[j], sum[0]);
        double total[1];
        row_sums<1, WAVE>(sum, total, lds);
        const RowScale r(row_scale(total[0], H, a.eps));
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const int64_t c = (int64_t)(tid + j * P) * VEC;
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) y[i] = r.times(h[j].at(i), w[j].at(i));
            if constexpr (FP8) {
                if ((int64_t)((tid & ~(kWave - 1)) + j * P) * VEC >= H) break;       // (the whole wave)
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const uint32_t u = __float_as_uint(y[i]) & 0x7FFFFFFFu;
                    m = u <= 0x7F800000u && u > m ? u : m;
                }
                m = dpp_umax_step<0x140>(half_row_umax(m));      // row_mirror: the other 8 of the group's 16 lanes
                const float amax = __uint_as_float(m);
                const Fp8Group q(amax, (a.flags & CDL_FP8_SCALE_UE8M0) != 0);
                const u32x2 code = quant8(y, q);
                store_scale(a, q, t, c / 128, (int64_t)((tid & ~(kWave - 1)) + j * P) * VEC / 128, c < H);
                if (c < H) *reinterpret_cast<u32x2 *>(a.q + row + c) = code;
            }
            if ((!FP8 || a.out) && c < H) {
                Unit<VEC> o;
                o.set(y);
                o.store(a.out + row + c);
            }
        }
    }
}

// Rows beyond kNormHeld columns: h is formed (and stored) in a first pass over
// the row and read again in the second, each element by the thread that wrote
// it.
template <int VEC, bool FP8>
__global__ __launch_bounds__(kNormThreads) void rms_norm_long_kernel(NormArgs a)
{
    __shared__ double lds[4];
    const int64_t H = a.H;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * H;
        double sum[1] = {0.0};
        for (int64_t c = (int64_t)threadIdx.x * VEC; c < H; c += kNormThreads * VEC) {
            Unit<VEC> h;
            h.load(a.x + row + c);
            if (a.res) {
                Unit<VEC> r;
                r.load(a.res + row + c);
                h.add(r);
                h.store(a.res_out + row + c);
            }
            sum[0] = add_squares(h, sum[0]);
        }
        double total[1];
        row_sums<1, false>(sum, total, lds);
        const RowScale r(row_scale(total[0], H, a.eps));
        const uint16_t *src = a.res ? a.res_out : a.x;
        for (int64_t c0 = 0; c0 < H; c0 += kNormThreads * VEC) {
            const int64_t c = c0 + (int64_t)threadIdx.x * VEC;
            const int64_t first = c0 + (int64_t)(threadIdx.x & ~(kWave - 1)) * VEC;
            if (first >= H) break;
            Unit<VEC> h, w;
            h.clear();
            w.clear();
            if (c < H) {
                h.load(src + row + c);
                w.load(a.w + c);
            }
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) y[i] = r.times(h.at(i), w.at(i));
            if constexpr (FP8) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const uint32_t u = __float_as_uint(y[i]) & 0x7FFFFFFFu;
                    m = u <= 0x7F800000u && u > m ? u : m;
                }
                m = dpp_umax_step<0x140>(half_row_umax(m));
                const float amax = __uint_as_float(m);
                const Fp8Group q(amax, (a.flags & CDL_FP8_SCALE_UE8M0) != 0);
                const u32x2 code = quant8(y, q);
                store_scale(a, q, t, c / 128, first / 128, c < H);
                if (c < H) *reinterpret_cast<u32x2 *>(a.q + row + c) = code;
            }
            if ((!FP8 || a.out) && c < H) {
                Unit<VEC> o;
                o.set(y);
                o.store(a.out + row + c);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// gradient: with n = h r and d = dy w,
//   dx = r (d - n mean(d n)) + dh,   dweight[c] = sum over rows of dy n
//
// A workgroup takes every G-th row and keeps its threads' columns of dweight in
// registers; the G partial sums go to the workspace and a second kernel adds
// them in order.  The next row's loads are under way while a row is summed.
// 16384 x 4096 with residual: 103 to 112 us (537 MB, 4.8 to 5.2 TB/s), the sums 5
// us of them.  Units of 1: 4096 x 7167 184 us against 44.  A narrow row still
// takes a workgroup, two barriers and most of its threads idle: 16384 x 512 45 us
// (1.5 TB/s), 200000 x 64 470 us (0.2 TB/s).
// ---------------------------------------------------------------------------
struct NormGradArgs {
    const uint16_t *dy, *h, *w, *dres;
    float eps;
    int64_t T, H;
    uint16_t *dx;
    float *dweight;
    float *partial;              // [G, H]
    float2 *stats;               // long rows: [T] (r, r^3 mean(d h))
    int32_t G;
};

// s + a unit's sums of h^2 and d h, in 64 bits as the norm's.
template <int VEC>
__device__ __forceinline__ void add_gradient_sums(const Unit<VEC> &h, const Unit<VEC> &g, const Unit<VEC> &w, double (&s)[2])
{
    s[0] = add_squares(h, s[0]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[1] = fma((double)(g.at(i) * w.at(i)), (double)h.at(i), s[1]);
}

template <int VEC, int NU>
__global__ __launch_bounds__(kNormThreads) void rms_norm_grad_kernel(NormGradArgs a)
{
    constexpr int P = kNormThreads;
    __shared__ double lds[8];
    const int tid = threadIdx.x;
    const int64_t H = a.H;
    Unit<VEC> w[NU], h[NU], g[NU];
    float acc[NU][VEC];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int64_t c = (int64_t)(tid + j * P) * VEC;
        w[j].clear();
        h[j].clear();
        g[j].clear();
        if (c < H) w[j].load(a.w + c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[j][i] = 0.0f;
    }
    auto load = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const int64_t c = (int64_t)(tid + j * P) * VEC;
            if (c < H) {
                h[j].load(a.h + t * H + c);
                g[j].load(a.dy + t * H + c);
            }
        }
    };
    if ((int64_t)blockIdx.x < a.T) load(blockIdx.x);
    for (int64_t t = blockIdx.x; t < a.T; t += a.G) {
        Unit<VEC> hh[NU], gg[NU], dr[NU];
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            hh[j] = h[j];
            gg[j] = g[j];
            dr[j].clear();
        }
        if (t + a.G < a.T) load(t + a.G);
        if (a.dres) {
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int64_t c = (int64_t)(tid + j * P) * VEC;
                if (c < H) dr[j].load(a.dres + t * H + c);
            }
        }
        double s[2] = {0.0, 0.0};
#pragma unroll
        for (int j = 0; j < NU; ++j) add_gradient_sums(hh[j], gg[j], w[j], s);
        double total[2];
        row_sums<2, false>(s, total, lds);
        const double rd = row_scale(total[0], H, a.eps);
        const float r = (float)rd, k = (float)(total[1] / (double)H * rd * rd);             // mean(d n) r, so that dx = r (d - h k)
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const int64_t c = (int64_t)(tid + j * P) * VEC;
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float x = hh[j].at(i), d = gg[j].at(i);
                o[i] = fmaf(r, fmaf(-x, k, d * w[j].at(i)), dr[j].at(i));
                acc[j][i] = fmaf(d, x * r, acc[j][i]);
            }
            Unit<VEC> u;
            u.set(o);
            if (c < H) u.store(a.dx + t * H + c);
        }
    }
#pragma unroll
    for (int j = 0; j < NU; ++j) {
        const int64_t c = (int64_t)(tid + j * P) * VEC;
        if (c < H) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) a.partial[(int64_t)blockIdx.x * H + c + i] = acc[j][i];
        }
    }
}

// Long rows: every row's two numbers, then the elements by blocks of columns
// (grid.x) and slices of rows (grid.y of them).
template <int VEC>
__global__ __launch_bounds__(kNormThreads) void rms_norm_grad_stats_kernel(NormGradArgs a)
{
    __shared__ double lds[8];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        double s[2] = {0.0, 0.0};
        for (int64_t c = (int64_t)threadIdx.x * VEC; c < a.H; c += kNormThreads * VEC) {
            Unit<VEC> h, g, w;
            h.load(a.h + t * a.H + c);
            g.load(a.dy + t * a.H + c);
            w.load(a.w + c);
            add_gradient_sums(h, g, w, s);
        }
        double total[2];
        row_sums<2, false>(s, total, lds);
        const double r = row_scale(total[0], a.H, a.eps);
        if (threadIdx.x == 0) a.stats[t] = float2{(float)r, (float)(total[1] / (double)a.H * r * r)};
    }
}

template <int VEC>
__global__ __launch_bounds__(kNormThreads) void rms_norm_grad_columns_kernel(NormGradArgs a)
{
    const int64_t c = ((int64_t)blockIdx.x * kNormThreads + threadIdx.x) * VEC;
    if (c >= a.H) return;
    Unit<VEC> w;
    w.load(a.w + c);
    float acc[VEC] = {};
    for (int64_t t = blockIdx.y; t < a.T; t += a.G) {
        const float2 s = a.stats[t];
        Unit<VEC> h, g, dr, u;
        h.load(a.h + t * a.H + c);
        g.load(a.dy + t * a.H + c);
        dr.clear();
        if (a.dres) dr.load(a.dres + t * a.H + c);
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float x = h.at(i), d = g.at(i);
            o[i] = fmaf(s.x, fmaf(-x, s.y, d * w.at(i)), dr.at(i));
            acc[i] = fmaf(d, x * s.x, acc[i]);
        }
        u.set(o);
        u.store(a.dx + t * a.H + c);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) a.partial[(int64_t)blockIdx.y * a.H + c + i] = acc[i];
}

// dweight from the G partial sums: 32 columns a workgroup, 32 slices of G
// summed side by side (8 loads under way each), then those in order.
constexpr int kDwColumns = 32, kDwSlices = 32;
__global__ __launch_bounds__(1024) void rms_norm_dweight_kernel(const float *__restrict__ partial, int G, int64_t H,
                                                                float *__restrict__ dweight)
{
    __shared__ float lds[kDwSlices][kDwColumns];
    const int col = threadIdx.x % kDwColumns, slice = threadIdx.x / kDwColumns;
    const int64_t c = (int64_t)blockIdx.x * kDwColumns + col;
    float s = 0.0f;
    if (c < H) {
#pragma unroll 8
        for (int b = slice; b < G; b += kDwSlices) s += partial[(int64_t)b * H + c];
    }
    lds[slice][col] = s;
    __syncthreads();
    if (slice == 0 && c < H) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kDwSlices; ++i) v += lds[i][col];
        dweight[c] = v;
    }
}

// ---------------------------------------------------------------------------
// fp8 outside a scatter
// ---------------------------------------------------------------------------

// One block of 128 x 128 weights per workgroup: 16 lanes take a row's 128, a
// thread 8 rows.  32 x 4096 x 7168: 516 us (2.8 GB, 5.5 TB/s).
__global__ __launch_bounds__(256) void quant_fp8_blocks_kernel(const uint16_t *__restrict__ w, int64_t N, int64_t K, int64_t NB,
                                                               int64_t G, int64_t blocks, uint8_t *__restrict__ q,
                                                               float *__restrict__ s)
{
    __shared__ uint32_t lds[4];
    for (int64_t id = blockIdx.x; id < blocks; id += gridDim.x) {
        const int64_t g = id % G, nb = id / G % NB, mat = id / G / NB;
        const int r0 = threadIdx.x >> 4, lane16 = threadIdx.x & 15;
        const int64_t base = (mat * N + nb * 128) * K + g * 128 + lane16 * 8;
        Unit<8> u[8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i].clear();
            if (nb * 128 + r0 + 16 * i < N) u[i].load(w + base + (r0 + 16 * i) * K);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t x = __float_as_uint(u[i].at(j)) & 0x7FFFFFFFu;
                m = x <= 0x7F800000u && x > m ? x : m;
            }
        }
#pragma unroll
        for (int x = 1; x < kWave; x *= 2) {
            const uint32_t o = (uint32_t)__shfl_xor((int)m, x);
            m = m > o ? m : o;
        }
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) m = m > lds[i] ? m : lds[i];
        const Fp8Group f(__uint_as_float(m), false);
        if (threadIdx.x == 0) s[id] = f.scale;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (nb * 128 + r0 + 16 * i < N)
                *reinterpret_cast<u32x2 *>(q + base + (r0 + 16 * i) * K) = quant8(
                    {u[i].at(0), u[i].at(1), u[i].at(2), u[i].at(3), u[i].at(4), u[i].at(5), u[i].at(6), u[i].at(7)}, f);
        __syncthreads();
    }
}

// 16 codes a thread, 8 threads a group.
__global__ __launch_bounds__(256) void dequant_fp8_kernel(const uint8_t *__restrict__ q, const uint32_t *__restrict__ s,
                                                          ScaleWords sw, bool packed, int64_t rows, int64_t H, int64_t rpm,
                                                          uint16_t *__restrict__ out)
{
    const int64_t per = H / 16, n = rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per, u = i - row * per, g = u / 8;
        int64_t at = sw.row * row;
        if (sw.mat) at = row / rpm * sw.mat + row % rpm * sw.row;
        float p;
        if (packed) {
            const uint32_t c = s[at + g / 4 * sw.batch] >> (8 * (g & 3)) & 255u;
            p = __uint_as_float(c == 0 ? 0x00400000u : c == 255 ? 0x7FC00000u : c << 23);
        } else {
            p = __uint_as_float(s[at + g * (sw.group ? sw.group : 1)]);
        }
        const u32x4 v = *reinterpret_cast<const u32x4 *>(q + row * H + u * 16);
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[j], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[j], true);
            o[2 * j] = pack_bf16(lo[0] * p, lo[1] * p);
            o[2 * j + 1] = pack_bf16(hi[0] * p, hi[1] * p);
        }
        u32x4 *to = reinterpret_cast<u32x4 *>(out + row * H + u * 16);
        to[0] = u32x4{o[0], o[1], o[2], o[3]};
        to[1] = u32x4{o[4], o[5], o[6], o[7]};
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

inline int check_norm(int64_t T, int64_t H, float eps)
{
    if (T < 0 || H < 1 || !(eps >= 0.0f)) return CDL_ERR_BAD_SIZE;
    if (H > CDL_MAX_HIDDEN || T > INT32_MAX) return CDL_ERR_TOO_LARGE;
    return CDL_OK;
}

template <int VEC, bool FP8>
int launch_norm(const NormArgs &a, hipStream_t stream)
{
    const int64_t most = 1 << 22;        // workgroups; more rows go around
    const dim3 rows((unsigned)(a.T < most ? a.T : most)), waves((unsigned)((a.T + 3) / 4 < most ? (a.T + 3) / 4 : most)),
        threads(kNormThreads);
    constexpr int U = 32 / VEC;          // units of the longest held row
    if (a.H > kNormHeld)
        rms_norm_long_kernel<VEC, FP8><<<rows, threads, 0, stream>>>(a);
    else if (a.H > kNormHeld / 2)
        rms_norm_kernel<VEC, U, false, FP8><<<rows, threads, 0, stream>>>(a);
    else if (a.H > kNormHeld / 4)
        rms_norm_kernel<VEC, U / 2, false, FP8><<<rows, threads, 0, stream>>>(a);
    else if (a.H > 1024)
        rms_norm_kernel<VEC, U / 4, false, FP8><<<rows, threads, 0, stream>>>(a);
    else if (a.H > 512)
        rms_norm_kernel<VEC, U / 2, true, FP8><<<waves, threads, 0, stream>>>(a);
    else
        rms_norm_kernel<VEC, U / 4, true, FP8><<<waves, threads, 0, stream>>>(a);
    return launch_status();
}

// Workgroups of the gradient: two a CU.
constexpr int kNormGradWgs = 512;

inline int norm_grad_wgs(int64_t T) { return (int)(T < kNormGradWgs ? T : kNormGradWgs); }

inline size_t norm_grad_stats_bytes(int64_t T, int64_t H) { return H > kNormHeld ? ((size_t)T * 8 + 255) & ~(size_t)255 : 0; }

inline size_t norm_grad_ws_bytes(int64_t T, int64_t H)
{
    const size_t n = norm_grad_stats_bytes(T, H) + (size_t)norm_grad_wgs(T) * (size_t)H * 4;
    return n < 256 ? 256 : (n + 255) & ~(size_t)255;
}

template <int VEC>
int launch_norm_grad(const NormGradArgs &a, hipStream_t stream)
{
    const dim3 wgs((unsigned)a.G), threads(kNormThreads);
    constexpr int U = 32 / VEC;
    if (a.T > 0) {
        if (a.H > kNormHeld) {
            rms_norm_grad_stats_kernel<VEC><<<dim3((unsigned)(a.T < 65536 ? a.T : 65536)), threads, 0, stream>>>(a);
            int rc = launch_status();
            if (rc != CDL_OK) return rc;
            const int64_t cols = (a.H + VEC * kNormThreads - 1) / (VEC * kNormThreads);
            rms_norm_grad_columns_kernel<VEC><<<dim3((unsigned)cols, (unsigned)a.G), threads, 0, stream>>>(a);
        } else if (a.H > kNormHeld / 2) {
            rms_norm_grad_kernel<VEC, U><<<wgs, threads, 0, stream>>>(a);
        } else if (a.H > kNormHeld / 4) {
            rms_norm_grad_kernel<VEC, U / 2><<<wgs, threads, 0, stream>>>(a);
        } else {
            rms_norm_grad_kernel<VEC, U / 4><<<wgs, threads, 0, stream>>>(a);
        }
        int rc = launch_status();
        if (rc != CDL_OK) return rc;
    }
    rms_norm_dweight_kernel<<<dim3((unsigned)((a.H + kDwColumns - 1) / kDwColumns)), dim3(kDwColumns * kDwSlices), 0, stream>>>(a.partial, a.G, a.H, a.dweight);
    return launch_status();
}

inline bool vector_rows(int64_t H, std::initializer_list<const void *> rows)
{
    bool ok = H % 8 == 0;
    for (const void *p : rows) ok = ok && aligned(p, 16);
    return ok;
}

}  // namespace

extern "C" {

int cdl_rms_norm(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float eps, int64_t T, int64_t H,
                 uint16_t *out, uint16_t *residual_out, void *stream)
{
    int rc = check_norm(T, H, eps);
    if (rc != CDL_OK) return rc;
    if (T == 0) return CDL_OK;
    if (!residual) residual_out = nullptr;                   // (ignored, its alignment too)
    if (!x || !weight || !out || (residual && !residual_out)) return CDL_ERR_NULL_POINTER;
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(weight, 2) || !aligned(out, 2) || !aligned(residual_out, 2))
        return CDL_ERR_UNSUPPORTED;
    const NormArgs a = {x, residual, weight, eps, T, H, out, residual_out, nullptr, nullptr, 0, ScaleWords(0, 0, 0, false, 0)};
    return vector_rows(H, {x, residual, weight, out, residual_out}) ? launch_norm<8, false>(a, (hipStream_t)stream)
                                                                    : launch_norm<1, false>(a, (hipStream_t)stream);
}

int cdl_rms_norm_fp8(const uint16_t *x, const uint16_t *residual, const uint16_t *weight, float eps, int64_t T, int64_t H,
                     uint8_t *out_q, void *out_scales, int32_t scale_flags, uint16_t *out, uint16_t *residual_out, void *stream)
{
    int rc = check_norm(T, H, eps);
    if (rc != CDL_OK) return rc;
    if (H % CDL_FP8_GROUP != 0 || !valid_scale_flags(scale_flags)) return CDL_ERR_UNSUPPORTED;
    if (T == 0) return CDL_OK;
    if (!residual) residual_out = nullptr;
    if (!x || !weight || !out_q || !out_scales || (residual && !residual_out)) return CDL_ERR_NULL_POINTER;
    if (!vector_rows(H, {x, residual, weight, out, residual_out}) || !aligned(out_q, 8) || !aligned(out_scales, 4))
        return CDL_ERR_UNSUPPORTED;
    const NormArgs a = {x,   residual,     weight, eps,        T,           H,
                        out, residual_out, out_q,  out_scales, scale_flags, ScaleWords(scale_flags, T, 0, false, H / CDL_FP8_GROUP)};
    return launch_norm<8, true>(a, (hipStream_t)stream);
}

size_t cdl_rms_norm_grad_workspace_size(int64_t T, int64_t H)
{
    return check_norm(T, H, 0.0f) == CDL_OK ? norm_grad_ws_bytes(T, H) : 0;
}

int cdl_rms_norm_grad(const uint16_t *dy, const uint16_t *h, const uint16_t *weight, const uint16_t *dresidual, float eps,
                      int64_t T, int64_t H, uint16_t *dx, float *dweight, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_norm(T, H, eps);
    if (rc != CDL_OK) return rc;
    if (!dweight || (T > 0 && (!dy || !h || !weight || !dx || !ws))) return CDL_ERR_NULL_POINTER;
    if (T > 0 && ws_bytes < norm_grad_ws_bytes(T, H)) return CDL_ERR_WORKSPACE;
    if (!aligned(dy, 2) || !aligned(h, 2) || !aligned(weight, 2) || !aligned(dresidual, 2) || !aligned(dx, 2) ||
        !aligned(dweight, 4) || !aligned(ws, 8))
        return CDL_ERR_UNSUPPORTED;
    NormGradArgs a = {};
    a.dy = dy;
    a.h = h;
    a.w = weight;
    a.dres = dresidual;
    a.eps = eps;
    a.T = T;
    a.H = H;
    a.dx = dx;
    a.dweight = dweight;
    a.stats = static_cast<float2 *>(ws);
    a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + norm_grad_stats_bytes(T, H));
    a.G = norm_grad_wgs(T);
    return vector_rows(H, {dy, h, weight, dresidual, dx}) ? launch_norm_grad<8>(a, (hipStream_t)stream)
                                                          : launch_norm_grad<1>(a, (hipStream_t)stream);
}

int cdl_quant_fp8_blocks(const uint16_t *w, int64_t mats, int64_t N, int64_t K, uint8_t *q, float *scales, void *stream)
{
    if (mats < 0 || N < 1 || K < 1) return CDL_ERR_BAD_SIZE;
    if (N > CDL_MAX_HIDDEN || K > CDL_MAX_HIDDEN) return CDL_ERR_TOO_LARGE;
    if (K % CDL_FP8_GROUP != 0) return CDL_ERR_UNSUPPORTED;
    const int64_t NB = (N + 127) / 128, G = K / 128;
    if (mats > INT32_MAX / (NB * G)) return CDL_ERR_TOO_LARGE;
    if (mats == 0) return CDL_OK;
    if (!w || !q || !scales) return CDL_ERR_NULL_POINTER;
    if (!aligned(w, 16) || !aligned(q, 8) || !aligned(scales, 4)) return CDL_ERR_UNSUPPORTED;
    const int64_t blocks = mats * NB * G, most = 1 << 22;
    quant_fp8_blocks_kernel<<<dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, (hipStream_t)stream>>>(
        w, N, K, NB, G, blocks, q, scales);
    return launch_status();
}

int cdl_dequant_fp8(const uint8_t *q, const void *scales, int32_t scale_flags, int64_t rows, int64_t H, int64_t rows_per_mat,
                    uint16_t *out, void *stream)
{
    if (rows < 0 || H < 1 || rows_per_mat < 0) return CDL_ERR_BAD_SIZE;
    if (H > CDL_MAX_HIDDEN || rows > INT32_MAX) return CDL_ERR_TOO_LARGE;
    if (H % CDL_FP8_GROUP != 0 || !valid_scale_flags(scale_flags)) return CDL_ERR_UNSUPPORTED;
    if (rows == 0) return CDL_OK;
    if (rows_per_mat < 1) return CDL_ERR_BAD_SIZE;
    if (!q || !scales || !out) return CDL_ERR_NULL_POINTER;
    if (!aligned(q, 16) || !aligned(scales, 4) || !aligned(out, 16)) return CDL_ERR_UNSUPPORTED;
    const ScaleWords w(scale_flags, rows, rows_per_mat, rows_per_mat < rows, H / CDL_FP8_GROUP);
    const int64_t n = rows * (H / 16), blocks = (n + 255) / 256;
    dequant_fp8_kernel<<<dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, (hipStream_t)stream>>>(
        q, static_cast<const uint32_t *>(scales), w, (scale_flags & CDL_FP8_SCALE_PACKED) != 0, rows, H, rows_per_mat, out);
    return launch_status();
}

}  // extern "C"
