// products.hip -- the products grouped by expert in bf16 and in fp8 (e4m3fn
// rows with a scale per 128 elements, weights with one per 128 x 128 block),
// their SwiGLU forms and the bf16 gradients, for MI355X (gfx950).  Included
// after experts.hip (same translation unit).

namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// One kernel for all of them: out[b, a] = sum over the depth of A[a] * B[b],
// an output column a and an output row b.
//
//   form  A (256 of a tile)        B (MT of a tile)          depth
//   kFwd  rows of W[e] (n)         token rows                K
//   kDx   columns of W[e] (k)      rows of dy                N
//   kDw   columns of x (k)         columns of dy (n)         the expert's rows
//
// Depth runs along a row's bytes for operands taken by rows and across rows
// for those taken by columns.
//
// One workgroup of 8 waves per CU walks its XCD's eighth of the tile list.  A
// stage of 128 bytes of depth (64 rows of it by columns) is loaded straight to
// LDS, one or two stages ahead of the matrix instructions, across tile borders.
// With few rows an expert the weights' bytes bound the product, with many the
// matrix instructions, at the rate that the card's power allows.
//
// Measured, one MI355X: 128 tokens over 32 of 256 experts, K = 7168, N = 4096,
// 306 us in bf16 and 160 in fp8 (6.0 and 5.8 TB/s); 131072 rows of 128 uneven
// experts, K = N = 4096, 3.8 to 4.2 ms and 2.4 to 2.6 ms (1.1 and 1.75 PFLOP/s; a
// library product of one such matrix 1.47 to 1.58 and 3.0), the matrix unit 66 and
// 48% busy at 1.65 and 1.9 GHz.  In bf16 it multiplies 12% more rows there than
// exist; of 3.87 ms, 3.70 are left without its stores, and 3.41 with every tile
// loading the same lines, which stay in the L2.
// ---------------------------------------------------------------------------
// The scale and codes of a group of 128 values in fp8 from its largest
// magnitude (over its values that are not NaN; infinite if one is): the
// dispatch's quantisation, of 32-bit values.
struct Fp8Group {
    float scale, inverse;
    int ex;                      // UE8M0: scale = 2^ex
    bool ue8m0, empty, fast;

    __device__ __forceinline__ Fp8Group(float amax, bool ue) : inverse(0.0f), ex(-127), ue8m0(ue), empty(!(amax > 0.0f)), fast(false)
    {
        if (ue8m0) {
            if (!empty) {
                int x = 0;
                const float m = frexpf(amax, &x);            // 448 = 0.875 * 2^9
                ex = amax == __builtin_huge_valf() ? 127 : x - 9 + (m > 0.875f ? 1 : 0);
                ex = ex < -127 ? -127 : ex;
            }
            scale = ldexpf(1.0f, ex);
        } else {
            scale = amax / 448.0f;                           // correctly rounded
            // The quotient by one reciprocal with a correction step, as the
            // dispatch's (3 instructions an element against the division's 10),
            // where it cannot leave fp32's range.
            // (one path for the whole wave)
            fast = __ballot(!(amax >= 0x1p-96f && amax < __builtin_huge_valf())) == 0;
            const float r = __builtin_amdgcn_rcpf(scale);
            inverse = fmaf(fmaf(-scale, r, 1.0f), r, r);
        }
    }
    __device__ __forceinline__ uint8_t exponent() const { return (uint8_t)(ex + 127); }
    // 4 W values to W words of codes.  A NaN quotient (or an infinite one, of a
    // power of two) takes the NaN code with x's sign.
    template <int W>
    __device__ __forceinline__ void codes(const float (&x)[4 * W], uint32_t (&out)[W]) const
    {
        float q[4 * W], sum = 0.0f;
        // one branch a call, the same for the wave
        if (fast) {
#pragma unroll
            for (int i = 0; i < 4 * W; ++i) {
                // (up to 448 + 2^-15, which the conversion takes to 448)
                const float t = x[i] * inverse;
                q[i] = fmaf(-fmaf(t, scale, -x[i]), inverse, t);
            }
        } else if (ue8m0) {
#pragma unroll
            for (int i = 0; i < 4 * W; ++i) q[i] = ldexpf(x[i], -ex);
        } else {
#pragma unroll
            for (int i = 0; i < 4 * W; ++i) {
                const float d = empty ? x[i] : x[i] / scale; // correctly rounded
                q[i] = d > 448.0f ? 448.0f : d < -448.0f ? -448.0f : d;
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * W; ++i) sum += q[i];
#pragma unroll
        for (int w = 0; w < W; ++w) out[w] = pack4_e4m3(q[4 * w], q[4 * w + 1], q[4 * w + 2], q[4 * w + 3]);
        // (finite if every term is, |q| <= 464)
        if (__builtin_expect(!__builtin_isfinite(sum), 0)) {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                out[w] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = q[4 * w + i];
                    const uint32_t nan = (__float_as_uint(x[4 * w + i]) >> 24 & 0x80u) | 0x7Fu;
                    out[w] |= (__builtin_isfinite(v) ? pack2_e4m3(v, 0.0f) & 0xFFu : nan) << (8 * i);
                }
            }
        }
    }
};

enum ProductForm { kFwd, kDx, kDw };
enum ProductEpilogue { kPlain, kSwiglu, kSwigluGrad };

struct ProductArgs {
    const uint8_t *a;
    const uint8_t *b;
    int64_t rows;                // token rows of the buffer
    int64_t K, N;                // weights [L, N, K] (SwiGLU: N = 2 I)
    int32_t L;
    const int32_t *counts;
    const int64_t *seg;          // NULL: expert e's rows start at e * cap
    int64_t cap;
    int32_t *status;
    uint16_t *out;
    const uint16_t *dh;          // SwiGLU gradient: [rows, I]
    // fp8
    const uint8_t *b_s;          // token scales in the format below
    const float *a_s;            // [L, ceil(N / 128), K / 128]
    int64_t s_row, s_batch;      // words from a row's scales to the next row's, to the next four groups'
    int64_t s_group;             // column-major fp32: words to the next group's; else 0
    int64_t s_mat;               // column-major, padded: words of one expert's matrix; else 0
    int32_t s_packed;            // exponent bytes, four groups a word
    int32_t s_flags;
    uint8_t *hq;                 // SwiGLU: [rows, I] e4m3fn and its scales in the same format
    void *hs;
    int64_t h_row, h_group, h_mat;   // words of hs: row to row, word of groups to word, expert's matrix to the next
};

constexpr int kProductThreads = 512;
constexpr int kProductNT = 256;          // A of a tile
constexpr int kProductWgs = 256;         // one per CU
constexpr int kLine = 128;               // bytes of a row per stage: 64 bf16, or the 128 elements of an fp8 scale
constexpr int kScaleRing = 3;            // batches (four stages' scales) in LDS: in use, loaded, and being left
constexpr uint32_t kFar = 0x80000000u;   // no tile operand reaches this offset: loads there read no memory and give zeros

__device__ __forceinline__ uint32_t lds_address(const uint8_t *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)p;
}

// Loads that go to LDS directly, lane l's 16 (4) bytes to `to` + 16 (4) * l.
// In assembly, because the compiler cannot tell the buffers of a ring apart and
// waits for every such load before any read of LDS; these are waited for with
// sync_stage().  They have no register output, and lanes out of range write
// zeros.  M0 holds the LDS address; nothing else here uses it.
__device__ __forceinline__ void dma16(u32x4 r, uint32_t off, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(r),
                 "s"(__builtin_amdgcn_readfirstlane((int)to)));
}
__device__ __forceinline__ void dma4(u32x4 r, uint32_t off, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(off), "s"(r),
                 "s"(__builtin_amdgcn_readfirstlane((int)to)));
}
// (the values are the same in all lanes)
__device__ __forceinline__ u32x4 scalar_rsrc(const uint8_t *base, uint32_t bytes)
{
    const uint64_t p = (uint64_t)base;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xFFFFu)),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), (uint32_t)kRsrcWord3};
}

// All but the wave's newest LEFT loads have arrived, its reads of LDS too, and
// so have every other wave's.
template <int LEFT>
__device__ __forceinline__ void sync_stage()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ void swap_rows16(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

template <bool FP8, ProductForm FORM, int MT>
struct ProductShape {
    // 8 waves, 2 parts of A by 4 of B: wave w has A's half w % 2, and of B's blocks
    // of 16 rows every fourth from w / 2 on, so that a tile's live rows are spread
    // evenly over the waves.
    static constexpr int WN = 2, WM = 4;
    static constexpr int NF = kProductNT / 16 / WN;      // 16-row fragments per wave
    static constexpr int MF = MT / 16 / WM;
    static constexpr bool kACols = FORM != kFwd, kBCols = FORM == kDw;
    // stages of each operand in LDS: what is multiplied, and one or two on their way
    static constexpr int kABufs = MT == 256 ? 2 : 3, kBBufs = MT >= 192 ? 2 : 3;
    static constexpr int kABuf = kProductNT * kLine, kBBuf = MT * kLine;
    static constexpr int kBBase = kABufs * kABuf;
    static constexpr int kMinStages = kABufs;
    // Loads per wave and stage, B's first.  When stage s + 1 has to be there, what
    // was loaded behind its A (of stage s + 1 - kABufs on) and behind its B may be
    // under way.
    static constexpr int kAUnits = 4, kBUnits = MT / 64, kUnits = kAUnits + kBUnits;
    static constexpr int kLeftA = (kABufs - 1) * kBUnits + (kABufs - 2) * kAUnits, kLeftB = (kBBufs - 1) * kUnits;
    static constexpr int kLeft = kLeftA < kLeftB ? kLeftA : kLeftB;
    static constexpr int kScaleBatch = MT * 16 + 256;    // token scales, then the weights'
    static constexpr int kScales = kBBase + kBBufs * kBBuf;
    static constexpr int kAmax = kScales + (FP8 ? kScaleRing * kScaleBatch : 0);
    static constexpr size_t kLds = kAmax + (FP8 ? WN * MT * 4 : 0);   // then the tile table
};

// 1 / (1 + exp(-x)).  The exponential is the instruction's, whose argument x
// log2(e) is rounded once (a relative error of |x| 2^-24 where the gate is far
// below zero, else less), the reciprocal within 1 ulp: both far below the
// rounding of the results.  A tile's epilogue takes them up to 128 times a lane:
// 30000 rows of 40 experts, K = 320, N = 2112, bf16 SwiGLU 65 us, 76 with the
// library's exponential and 88 with a division too (4096 rows, K = 7168: 350, 354,
// 354).
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// What one side of a tile loads in a stage.
struct ProductSide {
    const uint8_t *p;            // by rows: the tile's first row; by columns: depth row 0
    const uint8_t *p2;           // SwiGLU: the first up row
    uint32_t bytes;              // by rows: bytes of the tile's rows
    int64_t depth;               // by columns: rows
    uint32_t ld;                 // bytes of a row
    uint32_t off;                // the lane's offset in unit 0 of stage 0
};

// A tile of the output.
struct TileAt {
    int64_t row0, n0;            // its first row (kDw: of the expert's weights) and column
    int64_t begin, count;        // the expert's rows
    int64_t m0;                  // the tile's first of them
    int e, live_m, live_n, stages;
};

template <bool FP8, ProductForm FORM, ProductEpilogue EPI, int MT>
struct ProductWg {
    using S = ProductShape<FP8, FORM, MT>;
    static constexpr int kCols = EPI == kPlain ? kProductNT : kProductNT / 2;     // output columns of a tile
    static constexpr int NF = S::NF, MF = S::MF;
    static constexpr int R = FP8 ? 2 : 4, D = R - 1;           // fragments of A in registers, read ahead
    static_assert(NF % R == 0, "a fragment's registers do not depend on the stage");
    static constexpr bool kUpByUnit = EPI != kPlain;           // A's units alternate between gate and up rows
    // fp8 values multiplied as bf16 ones, which hold them exactly.  The fp8 instructions (of either depth) drop what
    // lies below 2^-13 of the largest of 8 neighbouring products; a result rounded to bf16 does not show it, but h,
    // quantised again, lands on other codes: of an expert step of 4096 tokens 0.16% of them, so 0.001%, and the step's
    // result is off by 0.0024 of 64 bits instead of 0.0026 (0.0017 without the bf16 rows between product and combine).
    // It costs half the matrix rate and a conversion: gate/up products of 131072 rows of 128 experts, K = N = 4096,
    // 2.75 -> 4.25 ms; of 4096 rows of 32 experts, K = 7168, 235 -> 345 us; of 128 such rows in the padded buffer
    // 165 -> 168 us.
    static constexpr bool kAsBf16 = FP8 && EPI == kSwiglu;
    static constexpr int kSteps = kAsBf16 ? 4 : FP8 ? 1 : 2;   // matrix instructions per pair of fragments and stage

    const ProductArgs a;
    const int32_t *const ends;
    const int tiles_m, tiles_n;
    const int32_t last, step;                // the workgroup's tiles
    uint8_t *const lds;
    const int tid, lane, wave, wn, wm;
    const uint32_t lds0;                     // LDS address of the buffers
    const uint32_t a_lane, b_lane;           // a lane's place in the wave's first fragments
    // operands being loaded
    ProductSide sa, sb;
    int32_t id_a, id_b;                      // tile, stage and stages that each operand loads next
    int stage_a, stages_a, stage_b, stages_b;
    const uint8_t *tok_s, *w_s;              // fp8: the tile's scales
    int live_rows, live_blocks;              // rows with scales; weight scale blocks
    uint32_t load_batch, batch;              // ring positions
    int buf_a, buf_b;                        // buffers of the stage being multiplied
    TileAt at, at_b, known;                  // the tile being multiplied, B's, the one described last
    int32_t known_id;

    // A tile under way, M fragments of B a wave.
    template <int M>
    struct Work {
        f32x4 acc[NF][M];
        i32x8 fa[R], fb[M];
        f32x4 part[M];                       // fp8: the sums of a stage of the A fragment before, and their scales
        float part_s[M];
        // a stage's fragments of B as bf16, converted once; where the registers do not hold all of them, the rest for
        // every fragment of A
        static constexpr int kHeld = M < 4 ? 4 : 2;
        v8bf16 wide[kAsBf16 ? M : 1][kHeld];
        v8bf16 av[2];                        // of A, converted one step ahead
    };

    __device__ __forceinline__ ProductWg(const ProductArgs &args, uint8_t *l, const int32_t *e, int tm, int tn, int32_t end,
                                         int32_t every)
        : a(args), ends(e), tiles_m(tm), tiles_n(tn), last(end), step(every), lds(l), tid(threadIdx.x), lane(tid & (kWave - 1)), wave(wave_id()), wn(wave % S::WN), wm(wave / S::WN),
          lds0(lds_address(l)), a_lane(fragment_lane<S::kACols>(wn * S::NF)), b_lane(fragment_lane<S::kBCols>(wm)),
          load_batch(0), batch(0), buf_a(0), buf_b(0), known_id(-1)
    {
    }

    // ---- loading ----

    // A lane's offset in unit 0: by rows, 8 lanes take the 128 bytes of a row,
    // 16-byte chunk c of row r going to chunk c ^ (r / 2 % 8), so that the
    // fragment reads (16 rows, one chunk) touch all 64 banks; by columns, 32
    // lanes take 512 bytes of a depth row, 32-byte block c of depth row d going
    // to block c ^ (d % 4 + 4 (d / 8 % 2)), so that the transposing reads of 32
    // lanes (8 depth rows, 32 bytes each) do.  Unit j is 64 LDS rows (16 depth
    // rows) further on, which leaves these unchanged.
    __device__ __forceinline__ uint32_t row_chunk() const { return (uint32_t)((lane & 7) ^ (((wave & 1) << 2 | lane >> 4) & 7)); }
    __device__ __forceinline__ uint32_t column_chunk() const
    {
        const int d = 2 * wave + (lane >> 5);
        return (uint32_t)((lane & 31) ^ (((d & 3) | (d >> 3 & 1) << 2) << 1));
    }

    __device__ __forceinline__ void side_by_rows(ProductSide &s, const uint8_t *p, int64_t ld, int live)
    {
        s.p = p;
        s.ld = (uint32_t)ld;
        s.bytes = (uint32_t)live * s.ld;
        s.off = (uint32_t)(wave * 8 + (lane >> 3)) * s.ld + row_chunk() * 16;
    }
    __device__ __forceinline__ void side_by_columns(ProductSide &s, const uint8_t *p, int64_t ld, int64_t depth, int64_t first)
    {
        s.p = p;
        s.ld = (uint32_t)ld;
        s.depth = depth;
        const uint32_t at = (uint32_t)first * 2 + column_chunk() * 16;
        s.off = at < s.ld ? (uint32_t)(2 * wave + (lane >> 5)) * s.ld + at : kFar;
    }

    // The loads of one stage, unit by unit.
    struct Units {
        u32x4 ra, ra2, rb;
        uint32_t a_off, b_off, a_to, b_to;
    };
    template <bool COLS>
    __device__ __forceinline__ u32x4 side_rsrc(const ProductSide &s, const uint8_t *p, int stage) const
    {
        if constexpr (COLS) {
            const int64_t d0 = (int64_t)stage * 64, left = s.depth - d0;
            return scalar_rsrc(p + d0 * s.ld, (uint32_t)(left <= 0 ? 0 : left < 64 ? left : 64) * s.ld);
        } else {
            return scalar_rsrc(p, s.bytes);
        }
    }
    template <bool COLS>
    __device__ __forceinline__ uint32_t side_off(const ProductSide &s, int stage) const
    {
        if constexpr (COLS) {
            return s.off;
        } else {
            const uint32_t k = (uint32_t)stage * kLine;
            return k + row_chunk() * 16 < s.ld ? s.off + k : kFar;
        }
    }
    __device__ __forceinline__ void load_b(Units &u, int j) const
    {
        dma16(u.rb, u.b_off, u.b_to + j * 8192);
        u.b_off += (S::kBCols ? 16 : 64) * sb.ld;
    }
    __device__ __forceinline__ void load_a(Units &u, int j) const
    {
        dma16(kUpByUnit && (j & 1) ? u.ra2 : u.ra, u.a_off, u.a_to + j * 8192);
        if (!kUpByUnit || (j & 1)) u.a_off += (S::kACols ? 16 : 64) * sa.ld;
    }

    // The scales of stages 4 q to 4 q + 3: a row's four words (or the word that
    // packs them) per lane, the weights' by wave 7.
    __device__ __forceinline__ void load_scales(int q)
    {
        const uint32_t to = lds0 + S::kScales + (load_batch % kScaleRing) * S::kScaleBatch;
        if (wave < MT / 64) {
            const int row = wave * 64 + lane;
            const uint8_t *p = tok_s + (int64_t)q * a.s_batch * 4;
            if (a.s_row == 1) {
                const u32x4 r0 = scalar_rsrc(p, (uint32_t)live_rows * 4);
                dma4(r0, (uint32_t)row * 4, to + wave * 256);
                if (a.s_group) {
                    const int64_t left = a.K / 128 - 4 * q;
#pragma unroll
                    for (int g = 1; g < 4; ++g)
                        dma4(scalar_rsrc(p + g * a.s_group * 4, left > g ? (uint32_t)live_rows * 4 : 0u), (uint32_t)row * 4,
                             to + g * (MT * 4) + wave * 256);
                }
            } else {
                const u32x4 r = scalar_rsrc(p, (uint32_t)live_rows > 0 ? (uint32_t)(live_rows * a.s_row - q * a.s_batch) * 4 : 0u);
                if (a.s_packed)
                    dma4(r, (uint32_t)row * (uint32_t)a.s_row * 4, to + wave * 256);
                else
                    dma16(r, (uint32_t)row * (uint32_t)a.s_row * 4, to + wave * 1024);
            }
        } else if (wave == 7) {
            const int64_t G = a.K / 128;
            const uint32_t step = (uint32_t)(EPI == kPlain ? G : a.N / 256 * G) * 4;
            const uint32_t bytes = live_blocks == 0 ? 0u : (uint32_t)((live_blocks - 1) * (int64_t)step + G * 4) - (uint32_t)q * 16;
            // lane 4 b + g: block b's scale of group g
            dma4(scalar_rsrc(w_s + (int64_t)q * 16, bytes), lane < 8 ? (uint32_t)(lane >> 2) * step + (uint32_t)(lane & 3) * 4 : kFar,
                 to + MT * 16);
        }
        ++load_batch;
    }

    // Begins the loads of each operand's next stage, A's to its buffer buf_a and
    // B's to buf_b.
    __device__ __forceinline__ void begin_b(Units &u, int buf)
    {
        if (stage_b == stages_b) {
            id_b += step;
            set_b();
        }
        if (FP8 && (stage_b & 3) == 0) load_scales(stage_b >> 2);
        u.rb = side_rsrc<S::kBCols>(sb, sb.p, stage_b);
        u.b_off = side_off<S::kBCols>(sb, stage_b);
        u.b_to = lds0 + S::kBBase + (uint32_t)buf * S::kBBuf + (uint32_t)wave * 1024;
        ++stage_b;
    }
    __device__ __forceinline__ void begin_a(Units &u, int buf)
    {
        if (stage_a == stages_a) {
            id_a += step;
            set_a();
        }
        u.ra = side_rsrc<S::kACols>(sa, sa.p, stage_a);
        if (kUpByUnit) u.ra2 = side_rsrc<S::kACols>(sa, sa.p2, stage_a);
        u.a_off = side_off<S::kACols>(sa, stage_a);
        u.a_to = lds0 + (uint32_t)buf * S::kABuf + (uint32_t)wave * 1024;
        ++stage_a;
    }
    __device__ __forceinline__ void load_all_b(int buf)
    {
        Units u;
        begin_b(u, buf);
#pragma unroll
        for (int j = 0; j < S::kBUnits; ++j) load_b(u, j);
    }
    __device__ __forceinline__ void load_all_a(int buf)
    {
        Units u;
        begin_a(u, buf);
#pragma unroll
        for (int j = 0; j < S::kAUnits; ++j) load_a(u, j);
    }
    // Before the first tile: everything but what the first stage's turn loads.
    __device__ __forceinline__ void start(int32_t id)
    {
        id_a = id_b = id;
        set_b();
        set_a();
#pragma unroll
        for (int x = 0; x < S::kABufs; ++x) {
            if (x < S::kBBufs) load_all_b(x);
            load_all_a(x);
        }
        // the first stage of both
        sync_stage<(S::kBBufs - 1) * S::kUnits + (S::kABufs - S::kBBufs) * S::kAUnits>();
    }

    // Tile `id`.  Both operands ask for it, one after the other; the second time
    // it is known.  Tiles of the weights' gradient run over the experts, each with
    // tiles_m x tiles_n of them whatever its count.
    __device__ __forceinline__ TileAt describe(int32_t id)
    {
        if (id == known_id) return known;
        known_id = id;
        GroupedTile g;
        if constexpr (FORM == kDw) {
            const int32_t per = tiles_m * tiles_n, local = id % per;
            g.e = id / per;
            g.n = local / tiles_m;
            g.m = local % tiles_m;
        } else {
            grouped_place(g, ends, a.L, tiles_n, id);
        }
        // scalar loads: nothing writes these arrays meanwhile
        using scalar_i32 = __attribute__((address_space(4))) const int32_t;
        using scalar_i64 = __attribute__((address_space(4))) const int64_t;
        const int64_t c = ((scalar_i32 *)(uintptr_t)a.counts)[g.e];
        const int64_t first = a.seg ? ((scalar_i64 *)(uintptr_t)a.seg)[g.e] : (int64_t)g.e * a.cap;
        bool bad;
        g.count = held_rows(a, c, first, &g.begin, &bad);
        TileAt t;
        t.e = g.e;
        t.begin = g.begin;
        t.count = g.count;
        if constexpr (FORM == kDw) {
            t.m0 = (int64_t)g.m * MT;
            t.live_m = (int)(a.N - t.m0 < MT ? a.N - t.m0 : MT);
        } else {
            // An expert's row tiles share its rows evenly: workgroups that read the same weights keep step, so
            // that all but the first find them in the L2.  131072 rows of 128 experts, K = N = 4096: full tiles and
            // a rest 51% of the requests, 4.25 ms; evenly in blocks of 64 rows 4.15 ms; evenly 76%, 4.02 ms.
            const int c = (int)g.count, tiles = (c + MT - 1) / MT, mt = tiles > 1 ? tiles : 1, q = c / mt, more = c - q * mt;
            const int m = g.m < mt ? g.m : mt - 1;
            t.m0 = (int64_t)m * q + (m < more ? m : more);
            t.live_m = q + (m < more ? 1 : 0);
        }
        t.n0 = (int64_t)g.n * kCols;
        t.row0 = FORM == kDw ? t.m0 : t.begin + t.m0;
        const int64_t cols = (FORM != kFwd ? a.K : EPI == kPlain ? a.N : a.N / 2) - t.n0;
        t.live_n = (int)(cols < kCols ? cols : kCols);
        t.stages = FORM == kFwd  ? (int)((a.K * (FP8 ? 1 : 2) + kLine - 1) / kLine)
                   : FORM == kDx ? (int)((a.N * 2 + kLine - 1) / kLine)
                                 : (int)((t.count + 63) / 64);
        // empty stages (which read no memory) up to the number of buffers: what is loaded is one tile ahead at most
        if (t.stages < S::kMinStages) t.stages = S::kMinStages;
        known = t;
        return t;
    }
    // Moves an operand to its next tile; past the last it is empty.
    __device__ __forceinline__ void set_a()
    {
        const bool none = id_a >= last;
        const TileAt t = describe(none ? last - 1 : id_a);
        stage_a = 0;
        stages_a = none ? INT32_MAX : t.stages;
        if constexpr (FORM == kDw) {
            side_by_columns(sa, a.a + t.begin * a.K * 2, a.K * 2, none ? 0 : t.count, t.n0);
        } else if constexpr (FORM == kDx) {
            side_by_columns(sa, a.a + (int64_t)t.e * a.N * a.K * 2, a.K * 2, none ? 0 : a.N, t.n0);
        } else {
            const int64_t row = a.K * (FP8 ? 1 : 2);
            side_by_rows(sa, a.a + ((int64_t)t.e * a.N + t.n0) * row, row, none ? 0 : t.live_n);
            sa.p2 = sa.p + a.N / 2 * row;
        }
    }
    __device__ __forceinline__ void set_b()
    {
        const bool none = id_b >= last;
        const TileAt t = describe(none ? last - 1 : id_b);
        at_b = t;
        stage_b = 0;
        stages_b = none ? INT32_MAX : t.stages;
        if constexpr (FORM == kDw) {
            side_by_columns(sb, a.b + t.begin * a.N * 2, a.N * 2, none ? 0 : t.count, t.row0);
        } else {
            const int64_t row = FORM == kDx ? a.N * 2 : a.K * (FP8 ? 1 : 2);
            side_by_rows(sb, a.b + t.row0 * row, row, none ? 0 : t.live_m);
        }
        if constexpr (FP8) {
            const int64_t G = a.K / 128, NB = (a.N + 127) / 128, blk = t.n0 / 128;
            w_s = reinterpret_cast<const uint8_t *>(a.a_s + ((int64_t)t.e * NB + blk) * G);
            live_blocks = none ? 0 : EPI != kPlain || NB - blk > 1 ? 2 : 1;
            live_rows = none ? 0 : t.live_m;
            tok_s = a.b_s + 4 * (a.s_mat ? t.e * a.s_mat + t.m0 : t.row0 * a.s_row);
        }
    }

    // ---- fragments ----
    //
    // A fragment is 16 rows (columns) of an operand and the whole stage of
    // depth: lane l has row l % 16 and 16-byte chunks l / 16 and l / 16 + 4 of
    // the stage's eight (by columns: the same depths).  The order of the depth
    // is free as long as both operands share it: one v_mfma 16x16x128 takes
    // all of it (fp8), two 16x16x32 a chunk each (bf16).  D has B's row l % 16
    // and, in register i, A's row 4 (l / 16) + i.
    template <bool COLS>
    __device__ __forceinline__ uint32_t fragment_lane(int first) const       // first: the wave's first fragment
    {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (COLS) {
            const uint32_t x = (uint32_t)((i >> 2) | (g & 1) << 2);
            return (uint32_t)(8 * g + (i >> 2)) * 512 + (((uint32_t)first ^ x) << 5) + (uint32_t)(i & 3) * 8;
        } else {
            return (uint32_t)(first * 16 + i) * kLine + (uint32_t)((g ^ (i >> 1)) << 4);
        }
    }
    // fragment f of the wave's, from the buffer that begins at `at`; by rows
    // the two chunks are 64 bytes apart, swizzled
    template <bool COLS>
    __device__ __forceinline__ u32x4 half_fragment(uint32_t at, uint32_t of_lane, int f, int half) const
    {
        if constexpr (COLS) {
            const uint32_t p = at + (of_lane ^ (uint32_t)(f << 5)) + (uint32_t)half * (32 * 512);
            auto tr = [&](int q) {
                using lds_i16x4 = __attribute__((address_space(3))) i16x4;
                return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(uintptr_t)(p + q * 512)));
            };
            const u32x2 x = tr(0), y = tr(4);
            return u32x4{x.x, x.y, y.x, y.y};
        } else {
            using lds_u32x4 = __attribute__((address_space(3))) const u32x4;
            return *(lds_u32x4 *)(uintptr_t)(at + (of_lane ^ (uint32_t)(half * 64)) + f * (16 * kLine));
        }
    }
    static __device__ __forceinline__ i32x8 join(const u32x4 &lo, const u32x4 &hi)
    {
        return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    }
    static __device__ __forceinline__ u32x4 half_of(const i32x8 &x, int half)
    {
        return half ? u32x4{(uint32_t)x[4], (uint32_t)x[5], (uint32_t)x[6], (uint32_t)x[7]}
                    : u32x4{(uint32_t)x[0], (uint32_t)x[1], (uint32_t)x[2], (uint32_t)x[3]};
    }
    __device__ __forceinline__ i32x8 a_fragment(int buf, int n) const
    {
        const uint32_t at = lds0 + (uint32_t)buf * S::kABuf;
        return join(half_fragment<S::kACols>(at, a_lane, n, 0), half_fragment<S::kACols>(at, a_lane, n, 1));
    }
    __device__ __forceinline__ u32x4 b_half(int buf, int m, int half) const
    {
        return half_fragment<S::kBCols>(lds0 + S::kBBase + (uint32_t)buf * S::kBBuf, b_lane, m * S::WM, half);
    }
    __device__ __forceinline__ i32x8 b_fragment(int buf, int m) const { return join(b_half(buf, m, 0), b_half(buf, m, 1)); }

    // fp8: scale of the lane's row of fragment m in stage s of the batch in use
    __device__ __forceinline__ float token_scale(int s, int m) const
    {
        const uint32_t p = lds0 + S::kScales + (batch % kScaleRing) * S::kScaleBatch;
        const uint32_t row = (uint32_t)((m * S::WM + wm) * 16 + (lane & 15));
        // a row's four words side by side, four rows of words, or one word a row
        const uint32_t at = p + row * (a.s_row != 1 && !a.s_packed ? 16u : 4u) +
                            (uint32_t)(s & 3) * (a.s_packed ? 0u : a.s_row == 1 ? MT * 4u : 4u);
        const uint32_t w = *(__attribute__((address_space(3))) const uint32_t *)(uintptr_t)at;
        const uint32_t c = (w >> (8 * (s & 3))) & 255u;
        const uint32_t e = c == 0 ? 0x00400000u : c == 255 ? 0x7FC00000u : c << 23;
        return __uint_as_float(a.s_packed ? e : w);
    }
    // of the wave's weight rows (SwiGLU: up = 0, 1 its gate, up rows)
    __device__ __forceinline__ float weight_scale(int s, int up) const
    {
        const uint8_t *p = lds + S::kScales + (batch % kScaleRing) * S::kScaleBatch + MT * 16;
        const int block = EPI == kPlain ? wn : up;
        return *reinterpret_cast<const float *>(p + block * 16 + (s & 3) * 4);
    }

    // 8 of a fragment's fp8 values (x = 0 to 3) as bf16; both operands of a product take the same x, so that the depths
    // agree.
    static __device__ __forceinline__ v8bf16 as_bf16(const i32x8 &f, int x, bool again = false)
    {
        typedef __bf16 v2bf16 __attribute__((ext_vector_type(2)));
        int lo = f[2 * x], hi = f[2 * x + 1];
        if (again) asm volatile("" : "+v"(lo), "+v"(hi));      // not the registers of an earlier conversion
        const v2bf16 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false),
                     b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true),
                     c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false),
                     d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
        return v8bf16{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    static __device__ __forceinline__ f32x4 mma(const i32x8 &x, const i32x8 &y, f32x4 c, int half)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf16, half_of(x, half)),
                                                       __builtin_bit_cast(v8bf16, half_of(y, half)), c, 0, 0, 0);
    }

    // Share of `total` items that follows instruction i of `of`.
    template <typename F>
    static __device__ __forceinline__ void share(int i, int of, int total, F &&f)
    {
#pragma unroll
        for (int x = 0; x < total; ++x)
            if (x * of / total == i) f(x);
    }

    // fp8: the waiting sums of A fragment n into acc.
    template <int M>
    static __device__ __forceinline__ void add_part(Work<M> &k, int n, int m)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) k.acc[n][m][i] = fmaf(k.part[m][i], k.part_s[m], k.acc[n][m][i]);
        // here, not where the compiler would gather the additions of all fragments (whose sums then fill the registers)
        asm volatile("" : "+v"(k.acc[n][m]));
    }

    // Stage s of the tile, in the buffers buf_a and buf_b, its first fragments in
    // registers; leaves the next stage's there and loads into the buffers.
    //
    // The order is fixed by hand: every matrix instruction is followed by a
    // share of the other work.  B's fragments are in registers from the stage's
    // beginning on: behind the first barrier B's buffer takes a later stage.  The
    // second barrier stands where the last A fragments are in registers, and the
    // next stage has arrived: behind it A's buffer takes a later stage, and the
    // next stage's fragments are read.  (All loads behind the second barrier:
    // 131072 rows of 128 experts, K = N = 4096, bf16, 4.02 ms.)  fp8: the sums of a
    // stage are scaled and added while the next fragment's are under way.
    template <int M>
    __device__ __forceinline__ void run_stage(Work<(M > 0 ? M : 1)> &k, int s)
    {
        const int next_a = buf_a + 1 == S::kABufs ? 0 : buf_a + 1, next_b = buf_b + 1 == S::kBBufs ? 0 : buf_b + 1;
        if constexpr (M == 0) {
            __builtin_amdgcn_s_barrier();
            load_all_b(buf_b);
            sync_stage<S::kLeft>();
            load_all_a(buf_a);
        } else {
            float sc[M], sc2[M];
            if constexpr (FP8) {
                const bool real = (int64_t)s * kLine < a.K;  // a stage past the row's end has no scales
                const float g = weight_scale(s, 0), u = EPI == kPlain ? 0.0f : weight_scale(s, 1);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float t = token_scale(s, m);
                    sc[m] = real ? t * g : 0.0f;
                    sc2[m] = real && EPI != kPlain ? t * u : 0.0f;
                }
            }
            Units u;
            // matrix instructions per fragment, between the barriers, after them
            constexpr int kPer = kSteps * M, kBetween = (NF - D - 1) * kPer, kAfter = D * kPer;
            static_assert(NF - D > 1, "steps between the barriers");
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                if (n == 1) {
                    begin_b(u, buf_b);
                    __builtin_amdgcn_s_barrier();
                }
                if (n == NF - D) {
                    begin_a(u, buf_a);
                    sync_stage<S::kLeft>();
                }
                k.fa[(n + D) % R] = a_fragment(n + D < NF ? buf_a : next_a, (n + D) % NF);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < kPer; ++x) {
                    const int m = x % M;
                    if constexpr (kAsBf16) {
                        constexpr int kHeld = Work<M>::kHeld;
                        const int q = x / M;
                        if (q == 0) add_part(k, (n + NF - 1) % NF, m);
                        if (n == 0 && x == 0) k.wide[0][0] = as_bf16(k.fb[0], 0);
                        const v8bf16 bv = q < kHeld ? k.wide[m][q] : as_bf16(k.fb[m], q, true);
                        k.part[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k.av[q & 1], bv, q == 0 ? f32x4{} : k.part[m], 0, 0, 0);
                        // behind the matrix instruction: what the next one, and the next step, take
                        if (m == 0) k.av[(q + 1) & 1] = as_bf16(k.fa[(q < 3 ? n : n + 1) % R], (q + 1) & 3);
                        if (n == 0 && x + 1 < kPer && (x + 1) / M < kHeld)
                            k.wide[(x + 1) % M][(x + 1) / M] = as_bf16(k.fb[(x + 1) % M], (x + 1) / M);
                        k.part_s[m] = n >= NF / 2 ? sc2[m] : sc[m];
                    } else if constexpr (FP8) {
                        add_part(k, (n + NF - 1) % NF, m);
                        k.part[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k.fa[n % R], k.fb[m], f32x4{}, 0, 0, 0, 0, 0, 0);
                        k.part_s[m] = EPI != kPlain && n >= NF / 2 ? sc2[m] : sc[m];
                    } else {
                        k.acc[n][m] = mma(k.fa[n % R], k.fb[m], k.acc[n][m], x / M);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    // B's registers take the next stage's as soon as they are used up
                    if (n == NF - 1) {
                        if constexpr (kAsBf16) {
                            if (x / M == (Work<M>::kHeld == 4 ? 0 : 3)) k.fb[m] = b_fragment(next_b, m);
                        } else if constexpr (FP8)
                            k.fb[m] = b_fragment(next_b, m);
                        else
                            k.fb[m] = x < M ? join(b_half(next_b, m, 0), half_of(k.fb[m], 1)) : join(half_of(k.fb[m], 0), b_half(next_b, m, 1));
                    }
                    if (n >= 1 && n < NF - D) share((n - 1) * kPer + x, kBetween, S::kBUnits, [&](int j) { load_b(u, j); });
                    if (n >= NF - D) share((n - (NF - D)) * kPer + x, kAfter, S::kAUnits, [&](int j) { load_a(u, j); });
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }

    // A tile's products into acc, M fragments of B a wave (none: only its share of
    // the loads).
    template <int M>
    __device__ __forceinline__ void run_tile()
    {
        Work<(M > 0 ? M : 1)> k;
        if constexpr (M > 0) {
#pragma unroll
            for (int i = 0; i < NF; ++i)
#pragma unroll
                for (int j = 0; j < M; ++j) k.acc[i][j] = f32x4{};
#pragma unroll
            for (int j = 0; j < D; ++j) k.fa[j] = a_fragment(buf_a, j);
#pragma unroll
            for (int j = 0; j < M; ++j) {
                k.fb[j] = b_fragment(buf_b, j);
                k.part[j] = f32x4{};
                k.part_s[j] = 0.0f;
            }
            if constexpr (kAsBf16) k.av[0] = as_bf16(k.fa[0], 0);
        }
        for (int s = 0; s < at.stages; ++s) {
            run_stage<M>(k, s);
            if (FP8 && ((s & 3) == 3 || s == at.stages - 1)) ++batch;
            buf_a = buf_a + 1 == S::kABufs ? 0 : buf_a + 1;
            buf_b = buf_b + 1 == S::kBBufs ? 0 : buf_b + 1;
        }
        if constexpr (M > 0 && FP8) {
#pragma unroll
            for (int m = 0; m < M; ++m) add_part(k, NF - 1, m);
        }
        if constexpr (FP8 && EPI == kSwiglu)
            store_tile_fp8<M>(k);
        else if constexpr (M > 0)
            store_tile(k);
    }

    // ---- results ----

    // Four blocks of 16 columns of the lane's row as bf16.  The lanes of a row
    // trade (a 4 x 4 transpose over the four lanes of a row, then the halves of
    // two blocks) so that each store writes 64 bytes in a run.
    __device__ __forceinline__ void store_blocks(const f32x4 (&v)[4], uint16_t *row, int cols, bool live, bool vector,
                                                 int lane) const
    {
        const int g = lane >> 4;
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo[j] = pack_bf16(v[j][0], v[j][1]);
            hi[j] = pack_bf16(v[j][2], v[j][3]);
        }
        if (!vector) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 16 * j + 4 * g + i;
                    if (live && c < cols) row[c] = (uint16_t)((i < 2 ? lo[j] : hi[j]) >> (16 * (i & 1)));
                }
            return;
        }
        uint32_t *w[2] = {lo, hi};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            swap_halves(w[h][0], w[h][2]);
            swap_halves(w[h][1], w[h][3]);
            swap_rows16(w[h][0], w[h][1]);
            swap_rows16(w[h][2], w[h][3]);
        }
        // block g: bytes 0-15 in lo, hi [0, 1], 16-31 in lo, hi [2, 3]
        swap_halves(lo[0], lo[2]);
        swap_halves(hi[0], hi[2]);
        swap_halves(lo[1], lo[3]);
        swap_halves(hi[1], hi[3]);
        const int c = 16 * (g & 1) + 8 * (g >> 1);
        if (live && c < cols) *reinterpret_cast<u32x4 *>(row + c) = u32x4{lo[0], hi[0], lo[1], hi[1]};
        if (live && c + 32 < cols) *reinterpret_cast<u32x4 *>(row + c + 32) = u32x4{lo[2], hi[2], lo[3], hi[3]};
    }

    template <int M>
    __device__ __forceinline__ void store_tile(const Work<M> &k)
    {
        const int64_t ld = FORM == kFwd ? (EPI == kSwiglu ? a.N / 2 : a.N) : a.K;
        const bool vector = ld % 8 == 0 && (EPI != kSwigluGrad || a.N / 2 % 8 == 0) && ((uintptr_t)a.out & 15) == 0;
        const int64_t I = a.N / 2;
        constexpr int H = EPI == kPlain ? NF : NF / 2;       // blocks of output columns
        uint16_t *const first = a.out + ((FORM == kDw ? (int64_t)at.e * a.N : 0) + at.row0) * ld + at.n0;
        // computed here, and not ahead of the tile and kept in registers that its sums need
        int lane = this->lane;
        asm volatile("" : "+v"(lane));
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int t = (m * S::WM + wm) * 16 + (lane & 15);
            const bool live = t < at.live_m;
#pragma unroll
            for (int q = 0; q < H / 4; ++q) {
                const int c = (wn * H + q * 4) * 16;
                uint16_t *row = first + t * ld + c;
                f32x4 v[4], w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (EPI == kPlain) {
                        v[j] = k.acc[q * 4 + j][m];
                    } else {
                        const f32x4 gate = k.acc[q * 4 + j][m], up = k.acc[H + q * 4 + j][m];
                        f32x4 d = {};
                        if constexpr (EPI == kSwigluGrad) {
                            const int col = c + 16 * j + 4 * (lane >> 4);
                            const uint16_t *p = a.dh + (at.row0 + t) * I + at.n0 + col;
                            if (live && ((I & 3) == 0 && ((uintptr_t)a.dh & 7) == 0)) {
                                if (col < at.live_n) {
                                    const u32x2 x = *reinterpret_cast<const u32x2 *>(p);
                                    d = f32x4{bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y)};
                                }
                            } else if (live) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (col + i < at.live_n) d[i] = __uint_as_float((uint32_t)p[i] << 16);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float s = sigmoid(gate[i]);
                            if constexpr (EPI == kSwiglu) {
                                v[j][i] = gate[i] * s * up[i];
                            } else {
                                v[j][i] = d[i] * up[i] * (s * (1.0f + gate[i] * (1.0f - s)));
                                w[j][i] = d[i] * (gate[i] * s);
                            }
                        }
                    }
                }
                store_blocks(v, row, at.live_n - c, live, vector, lane);
                if constexpr (EPI == kSwigluGrad) store_blocks(w, row + I, at.live_n - c, live, vector, lane);
                __builtin_amdgcn_sched_barrier(0);           // one group's temporaries at a time
            }
        }
    }

    // SwiGLU values in fp8: a tile's 128 columns are one group, so the waves
    // of a row exchange their largest magnitudes.  Every wave comes here.
    template <int M>
    __device__ __forceinline__ void store_tile_fp8(Work<(M > 0 ? M : 1)> &k)
    {
        constexpr int H = NF / 2;
        static_assert(H == 4, "a lane's 16 codes are one store");
        float *amax = reinterpret_cast<float *>(lds + S::kAmax);
        if constexpr (M > 0) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
                uint32_t top = 0;                            // magnitudes as integers, NaNs left out
#pragma unroll
                for (int j = 0; j < H; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float g = k.acc[j][m][i];
                        const float h = g * sigmoid(g) * k.acc[H + j][m][i];
                        k.acc[j][m][i] = h;
                        const uint32_t u = __float_as_uint(h) & 0x7FFFFFFFu;
                        top = u <= 0x7F800000u && u > top ? u : top;
                    }
                uint32_t o = top;
                swap_halves(top, o);
                top = top > o ? top : o;
                o = top;
                swap_rows16(top, o);
                top = top > o ? top : o;
                if (lane < 16) amax[wn * MT + (m * S::WM + wm) * 16 + lane] = __uint_as_float(top);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if constexpr (M == 0) return;
        const int64_t I = a.N / 2;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int t = (m * S::WM + wm) * 16 + (lane & 15);
            float am = amax[t];
#pragma unroll
            for (int x = 1; x < S::WN; ++x) am = fmaxf(am, amax[x * MT + t]);
            const Fp8Group q(am, (a.s_flags & CDL_FP8_SCALE_UE8M0) != 0);
            const bool live = t < at.live_m;
            const int64_t row = at.row0 + t;
            uint32_t w[H];
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const float h[4] = {k.acc[j][m][0], k.acc[j][m][1], k.acc[j][m][2], k.acc[j][m][3]};
                uint32_t c[1];
                q.template codes<1>(h, c);
                w[j] = c[0];
            }
            uint8_t *to = a.hq + row * I + at.n0 + wn * H * 16;
            const int g = lane >> 4;
            swap_halves(w[0], w[2]);
            swap_halves(w[1], w[3]);
            swap_rows16(w[0], w[1]);
            swap_rows16(w[2], w[3]);
            if (live) *reinterpret_cast<u32x4 *>(to + 16 * g) = u32x4{w[0], w[1], w[2], w[3]};
            if (live && lane < 16 && wn == 0) {
                const int64_t grp = at.n0 / 128;
                const int64_t r = a.h_mat ? at.e * a.h_mat + (at.m0 + t) * a.h_row : row * a.h_row;
                if (a.s_packed) {
                    uint8_t *word = static_cast<uint8_t *>(a.hs) + (r + grp / 4 * a.h_group) * 4;
                    word[grp % 4] = q.exponent();
                    if (grp == I / 128 - 1)
                        for (int64_t x = grp % 4 + 1; x < 4; ++x) word[x] = 0;
                } else
                    static_cast<float *>(a.hs)[r + grp * a.h_group] = q.scale;
            }
        }
    }
};

template <bool FP8, ProductForm FORM, ProductEpilogue EPI, int MT>
__global__ __launch_bounds__(kProductThreads) void product_kernel(ProductArgs a, int tiles_m, int tiles_n)
{
    using Wg = ProductWg<FP8, FORM, EPI, MT>;
    using S = ProductShape<FP8, FORM, MT>;
    extern __shared__ u32x4 lds4[];
    uint8_t *lds = reinterpret_cast<uint8_t *>(lds4);
    int32_t *ends = reinterpret_cast<int32_t *>(lds + S::kLds);
    // (kDw only checks the counts here: its tiles do not depend on them)
    const int32_t counted = grouped_tile_table<MT>(a, FORM == kDw ? 1 : tiles_n, ends);
    const int32_t total = FORM == kDw ? a.L * tiles_m * tiles_n : counted;
    const int32_t per = (total + 7) / 8, step = (int32_t)(gridDim.x / 8);
    const int32_t first = (int32_t)(blockIdx.x & 7) * per;
    const int32_t last = first + per < total ? first + per : total;
    int32_t id = first + (int32_t)(blockIdx.x >> 3);
    if (id >= last) return;
    __syncthreads();
    Wg w(a, lds, ends, tiles_m, tiles_n, last, step);
    w.start(id);
    for (; id < last; id += step) {
        w.at = w.at_b;                                       // (B is not yet past this tile)
        const bool busy = w.wm * 16 < w.at.live_m;           // the wave has a live row
        const int blocks = busy ? (w.at.live_m + 63) / 64 : 0;
        if (blocks == S::MF)
            w.template run_tile<S::MF>();
        else if (blocks == 0)
            w.template run_tile<0>();
        else if (blocks == 1)
            w.template run_tile<1>();
        else if (blocks == 2 || S::MF < 4)
            w.template run_tile<(S::MF > 2 ? 2 : 1)>();
        else
            w.template run_tile<(S::MF > 3 ? 3 : 1)>();
    }
    // nothing may be on its way to this workgroup's LDS when it ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// A tile's operands are addressed with 32-bit offsets: 256 rows of at most
// 2^22 bytes.
inline int check_product(int64_t rows, int64_t K, int32_t L, int64_t N, const int32_t *counts, const int64_t *seg, int64_t cap)
{
    if (rows < 0 || K < 1 || N < 1 || L < 1 || L > CDL_MAX_LOCAL_EXPERTS) return CDL_ERR_BAD_SIZE;
    if (!seg && (cap < 0 || rows != (int64_t)L * cap)) return CDL_ERR_BAD_SIZE;
    if (K > CDL_MAX_PRODUCT_WIDTH || N > CDL_MAX_PRODUCT_WIDTH || rows > INT32_MAX - 256) return CDL_ERR_TOO_LARGE;
    if (!counts) return CDL_ERR_NULL_POINTER;
    return CDL_OK;
}

template <bool FP8, ProductForm FORM, ProductEpilogue EPI, int MT>
int launch_product_tiles(const ProductArgs &a, hipStream_t stream)
{
    using S = ProductShape<FP8, FORM, MT>;
    constexpr int kCols = EPI == kPlain ? kProductNT : kProductNT / 2;
    const int64_t width = FORM == kFwd ? (EPI == kPlain ? a.N : a.N / 2) : a.K;
    const int64_t tiles_n = (width + kCols - 1) / kCols;
    int64_t tiles, tiles_m = 0;
    // tile numbers keep room for a workgroup's step past the last one
    if (FORM == kDw) {
        tiles_m = (a.N + MT - 1) / MT;
        if (tiles_m * tiles_n > (INT32_MAX - kProductWgs) / a.L) return CDL_ERR_TOO_LARGE;
        tiles = a.L * tiles_m * tiles_n;
    } else {
        const int64_t most = a.seg ? a.rows : a.cap;
        if ((most + MT - 1) / MT * tiles_n > (INT32_MAX - kProductWgs) / a.L) return CDL_ERR_TOO_LARGE;
        tiles = (a.seg ? a.rows / MT + a.L : (int64_t)a.L * ((a.cap + MT - 1) / MT)) * tiles_n;
    }
    const int64_t filled = (tiles + 7) / 8 * 8, wgs = filled ? filled : 8;       // (none: the counts' check)
    product_kernel<FP8, FORM, EPI, MT><<<dim3((unsigned)(wgs < kProductWgs ? wgs : kProductWgs)), dim3(kProductThreads),
                                         S::kLds + (size_t)a.L * sizeof(int32_t), stream>>>(a, (int)tiles_m, (int)tiles_n);
    return launch_status();
}

// Buffers of very many experts leave no room for their tile table beside the
// smaller tiles' third stage (fp8: 1216 experts at 192 rows); 256 rows fit all.
template <bool FP8, ProductForm FORM, int MT>
bool product_fits(int32_t L)
{
    constexpr size_t kLdsBytes = 160 * 1024;
    static_assert(ProductShape<FP8, FORM, 256>::kLds + CDL_MAX_LOCAL_EXPERTS * sizeof(int32_t) <= kLdsBytes, "largest tile");
    return ProductShape<FP8, FORM, MT>::kLds + (size_t)L * sizeof(int32_t) <= kLdsBytes;
}

// Rows of a tile, 128, 192 or 256: the fewest rounds of the workgroups, weighed
// by what a round costs (1.03, 1.33 and 1.59 us a stage where the matrix
// instructions bound it).  The host sees the rows of the whole buffer only: an
// expert is taken to have their average, in one tile where that fills four
// fifths of it, otherwise half a tile more; a second round counts whole.  Measured, us for 128 / 192 / 256
// rows, bf16, 32 experts, K = 7168, N = 4096: 94 rows an expert 338 / 339 / 362,
// 128 rows 403 / 354 / 373, 172 rows 515 / 430 / 395, 256 rows 623 / 603 / 559,
// 512 rows 1042 / 942 / 892; 4 experts of 512 rows, K = N = 4096: 121 / 85 / 99;
// one of 4096 rows: 138 / 159 / 112; 8 of 250 rows, K = N = 1024: 21 / 26 / 30.
// Padded buffers are mostly empty in decode, where the weights' bytes count
// and three stages of them in LDS pay: 4 rows an expert, 32 experts, K = 7168,
// N = 4096, bf16 307 / 307 / 328, fp8 162 / 161 / 175.  A full one loses by it:
// 32 experts of 512 rows, K = N = 4096, bf16, 540 us at 192 rows, as segments (256)
// 455.  A buffer of eight times the rows (the average is then no expert's) does not:
// 4096 rows of 32 experts, K = 7168, SwiGLU, 361 us at 256 rows and 360 at 192.
template <bool FP8, ProductForm FORM, ProductEpilogue EPI>
int product_tile_rows(const ProductArgs &a)
{
    if (!a.seg) return product_fits<FP8, FORM, 192>(a.L) ? 192 : 256;
    const int64_t width = FORM == kDx ? a.K : EPI == kPlain ? a.N : a.N / 2, cols = EPI == kPlain ? kProductNT : kProductNT / 2;
    const double tiles_n = (double)((width + cols - 1) / cols), r = (double)a.rows / a.L;
    int best = 256;
    double least = 1e300;
    // Quantised SwiGLU takes 256 rows only where nothing else fits: their bf16 fragments do not (131072 rows of 128
    // experts, K = N = 4096: 128 / 192 / 256 rows 4.97 / 4.25 / 5.73 ms).
    constexpr int kMost = FP8 && EPI == kSwiglu ? 192 : 256;
    for (int mt = product_fits<FP8, FORM, kMost>(a.L) ? kMost : 256; mt >= 128; mt -= 64) {
        if (mt == 192 ? !product_fits<FP8, FORM, 192>(a.L) : mt == 128 && !product_fits<FP8, FORM, 128>(a.L)) continue;
        const double tm = a.L == 1 ? (double)((a.rows + mt - 1) / mt) : r <= 0.8 * mt ? 1.0 : r / mt + 0.5;
        const double rounds = tm * a.L * tiles_n / kProductWgs;
        const double cost = (rounds <= 1.0 ? 1.0 : rounds <= 2.0 ? 2.0 : rounds) * (mt == 128 ? 1.03 : mt == 192 ? 1.33 : 1.59);
        if (cost < least) {
            best = mt;
            least = cost;
        }
    }
    return best;
}

template <bool FP8, ProductForm FORM, ProductEpilogue EPI>
int launch_product(const ProductArgs &a, hipStream_t stream)
{
    if constexpr (FORM == kDw) {
        return launch_product_tiles<FP8, FORM, EPI, 256>(a, stream);
    } else {
        // (an empty buffer: only the check of the counts is left)
        if (a.rows == 0 && !a.status) return CDL_OK;
        const int mt = product_tile_rows<FP8, FORM, EPI>(a);
        return mt == 256   ? launch_product_tiles<FP8, FORM, EPI, 256>(a, stream)
               : mt == 192 ? launch_product_tiles<FP8, FORM, EPI, 192>(a, stream)
                           : launch_product_tiles<FP8, FORM, EPI, 128>(a, stream);
    }
}

inline ProductArgs product_args(const void *a, const void *b, int64_t rows, int64_t K, int32_t L, int64_t N,
                                const int32_t *counts, const int64_t *seg, int64_t cap, uint16_t *out, int32_t *status)
{
    ProductArgs p = {};
    p.a = static_cast<const uint8_t *>(a);
    p.b = static_cast<const uint8_t *>(b);
    p.rows = rows;
    p.K = K;
    p.L = L;
    p.N = N;
    p.counts = counts;
    p.seg = seg;
    p.cap = cap;
    p.out = out;
    p.status = status;
    return p;
}

// The words of a scale buffer of `rows` rows and G groups (padded buffers:
// cap rows a matrix where it is column-major).
struct ScaleWords {
    int64_t row, batch, group, mat;
    ScaleWords(int32_t flags, int64_t rows, int64_t cap, bool padded, int64_t G)
    {
        const bool packed = (flags & CDL_FP8_SCALE_PACKED) != 0;
        const int64_t words = packed ? (G + 3) / 4 : G;
        group = mat = 0;
        if (flags & CDL_FP8_SCALE_COLMAJOR) {
            const int64_t ld = ((padded ? cap : rows) + 3) / 4 * 4;
            row = 1;
            batch = packed ? ld : 4 * ld;
            group = packed ? 0 : ld;
            mat = padded ? words * ld : 0;
        } else {
            row = words;
            batch = packed ? 1 : 4;
        }
    }
};

inline int check_fp8_product(const uint8_t *q, const void *s, const uint8_t *wq, const float *ws, int64_t rows, int64_t K,
                             int32_t flags)
{
    if (!wq || !ws || (rows > 0 && (!q || !s))) return CDL_ERR_NULL_POINTER;
    if (K % CDL_FP8_GROUP != 0 || !valid_scale_flags(flags)) return CDL_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(wq, 16) || !aligned(s, 4) || !aligned(ws, 4)) return CDL_ERR_UNSUPPORTED;
    return CDL_OK;
}

inline void set_fp8(ProductArgs &p, const void *s, const float *ws, int32_t flags)
{
    const ScaleWords w(flags, p.rows, p.cap, p.seg == nullptr, p.K / CDL_FP8_GROUP);
    p.b_s = static_cast<const uint8_t *>(s);
    p.a_s = ws;
    p.s_row = w.row;
    p.s_batch = w.batch;
    p.s_group = w.group;
    p.s_mat = w.mat;
    p.s_packed = (flags & CDL_FP8_SCALE_PACKED) != 0;
    p.s_flags = flags;
}

}  // namespace

extern "C" {

int cdl_grouped_bf16(const uint16_t *x, int64_t rows, int64_t K, const uint16_t *w, int32_t L, int64_t N,
                     const int32_t *counts, const int64_t *seg_indptr, int64_t cap, uint16_t *out, int32_t *status,
                     void *stream)
{
    int rc = check_product(rows, K, L, N, counts, seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (!w || (rows > 0 && (!x || !out))) return CDL_ERR_NULL_POINTER;
    if (K % 8 != 0 || !aligned(x, 16) || !aligned(w, 16) || !aligned(out, 2)) return CDL_ERR_UNSUPPORTED;
    return launch_product<false, kFwd, kPlain>(product_args(w, x, rows, K, L, N, counts, seg_indptr, cap, out, status),
                                               (hipStream_t)stream);
}

int cdl_grouped_swiglu_bf16(const uint16_t *x, int64_t rows, int64_t K, const uint16_t *w, int32_t L, int64_t I,
                            const int32_t *counts, const int64_t *seg_indptr, int64_t cap, uint16_t *out, int32_t *status,
                            void *stream)
{
    int rc = check_product(rows, K, L, I < 1 ? I : 2 * (I < CDL_MAX_PRODUCT_WIDTH ? I : CDL_MAX_PRODUCT_WIDTH), counts,
                           seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (!w || (rows > 0 && (!x || !out))) return CDL_ERR_NULL_POINTER;
    if (K % 8 != 0 || !aligned(x, 16) || !aligned(w, 16) || !aligned(out, 2)) return CDL_ERR_UNSUPPORTED;
    return launch_product<false, kFwd, kSwiglu>(product_args(w, x, rows, K, L, 2 * I, counts, seg_indptr, cap, out, status),
                                                (hipStream_t)stream);
}

int cdl_grouped_swiglu_bf16_grad(const uint16_t *x, int64_t rows, int64_t K, const uint16_t *w, int32_t L, int64_t I,
                                 const uint16_t *dh, const int32_t *counts, const int64_t *seg_indptr, int64_t cap,
                                 uint16_t *out, int32_t *status, void *stream)
{
    int rc = check_product(rows, K, L, I < 1 ? I : 2 * (I < CDL_MAX_PRODUCT_WIDTH ? I : CDL_MAX_PRODUCT_WIDTH), counts,
                           seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (!w || (rows > 0 && (!x || !dh || !out))) return CDL_ERR_NULL_POINTER;
    if (K % 8 != 0 || !aligned(x, 16) || !aligned(w, 16) || !aligned(dh, 2) || !aligned(out, 2)) return CDL_ERR_UNSUPPORTED;
    ProductArgs a = product_args(w, x, rows, K, L, 2 * I, counts, seg_indptr, cap, out, status);
    a.dh = dh;
    return launch_product<false, kFwd, kSwigluGrad>(a, (hipStream_t)stream);
}

int cdl_grouped_bf16_dx(const uint16_t *dy, int64_t rows, int64_t N, const uint16_t *w, int32_t L, int64_t K,
                        const int32_t *counts, const int64_t *seg_indptr, int64_t cap, uint16_t *dx, int32_t *status,
                        void *stream)
{
    int rc = check_product(rows, K, L, N, counts, seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (!w || (rows > 0 && (!dy || !dx))) return CDL_ERR_NULL_POINTER;
    if (K % 8 != 0 || N % 8 != 0 || !aligned(dy, 16) || !aligned(w, 16) || !aligned(dx, 16)) return CDL_ERR_UNSUPPORTED;
    return launch_product<false, kDx, kPlain>(product_args(w, dy, rows, K, L, N, counts, seg_indptr, cap, dx, status),
                                              (hipStream_t)stream);
}

int cdl_grouped_bf16_dw(const uint16_t *dy, const uint16_t *x, int64_t rows, int64_t N, int64_t K, int32_t L,
                        const int32_t *counts, const int64_t *seg_indptr, int64_t cap, uint16_t *dw, int32_t *status,
                        void *stream)
{
    int rc = check_product(rows, K, L, N, counts, seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (!dw || (rows > 0 && (!dy || !x))) return CDL_ERR_NULL_POINTER;
    if (K % 8 != 0 || N % 8 != 0 || !aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16)) return CDL_ERR_UNSUPPORTED;
    return launch_product<false, kDw, kPlain>(product_args(x, dy, rows, K, L, N, counts, seg_indptr, cap, dw, status),
                                              (hipStream_t)stream);
}

int cdl_grouped_fp8(const uint8_t *q, const void *scales, int32_t scale_flags, int64_t rows, int64_t K, const uint8_t *w_q,
                    const float *w_scales, int32_t L, int64_t N, const int32_t *counts, const int64_t *seg_indptr,
                    int64_t cap, uint16_t *out, int32_t *status, void *stream)
{
    int rc = check_product(rows, K, L, N, counts, seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (rows > 0 && !out) return CDL_ERR_NULL_POINTER;
    rc = check_fp8_product(q, scales, w_q, w_scales, rows, K, scale_flags);
    if (rc != CDL_OK) return rc;
    if (!aligned(out, 2)) return CDL_ERR_UNSUPPORTED;
    ProductArgs a = product_args(w_q, q, rows, K, L, N, counts, seg_indptr, cap, out, status);
    set_fp8(a, scales, w_scales, scale_flags);
    return launch_product<true, kFwd, kPlain>(a, (hipStream_t)stream);
}

int cdl_grouped_swiglu_fp8(const uint8_t *q, const void *scales, int32_t scale_flags, int64_t rows, int64_t K,
                           const uint8_t *w_q, const float *w_scales, int32_t L, int64_t I, const int32_t *counts,
                           const int64_t *seg_indptr, int64_t cap, uint8_t *out_q, void *out_scales, int32_t *status,
                           void *stream)
{
    int rc = check_product(rows, K, L, I < 1 ? I : 2 * (I < CDL_MAX_PRODUCT_WIDTH ? I : CDL_MAX_PRODUCT_WIDTH), counts,
                           seg_indptr, cap);
    if (rc != CDL_OK) return rc;
    if (rows > 0 && (!out_q || !out_scales)) return CDL_ERR_NULL_POINTER;
    rc = check_fp8_product(q, scales, w_q, w_scales, rows, K, scale_flags);
    if (rc != CDL_OK) return rc;
    if (I % CDL_FP8_GROUP != 0 || !aligned(out_q, 16) || !aligned(out_scales, 4)) return CDL_ERR_UNSUPPORTED;
    ProductArgs a = product_args(w_q, q, rows, K, L, 2 * I, counts, seg_indptr, cap, nullptr, status);
    set_fp8(a, scales, w_scales, scale_flags);
    const ScaleWords h(scale_flags, rows, cap, seg_indptr == nullptr, I / CDL_FP8_GROUP);
    a.hq = out_q;
    a.hs = out_scales;
    a.h_row = h.row;
    a.h_group = a.s_packed ? h.batch : h.group ? h.group : 1;
    a.h_mat = h.mat;
    return launch_product<true, kFwd, kSwiglu>(a, (hipStream_t)stream);
}

}  // extern "C"
