// Attention over the 4-bit paged cache: new tokens of many requests (one
// each when decoding) against all positions their request holds.
//
// Mathematics.  With a code n, K = z + n s per 64-channel group, so
//   q . K = sum_g s_g * (q . n)_g + z_g * (sum of q)_g
//   sum_j p_j V_j = sum_j (p_j s_j) n_j + sum_j p_j z_j
// and only (q . n) and (p s) . n are matrix products, with the 4-bit codes as
// one operand.  The step is not applied to the codes but to the product (K)
// and to the weight (V), so unpacking is all that happens to a code.
//
// bf16: the bits 0000 0000 0000 nnnn are the fp16 number n 2^-24, and 0000
// 0000 nnnn 0000 is 16 n 2^-24 (subnormal, exact), so masks turn a word of
// codes into four fp16x2 operands: 5 integer instructions for 8 codes.  The
// factors go into the other operand (queries) or the result (values).
// Queries enter fp16 scaled by a power of two that brings their largest to
// 2^14 .. 2^15: bf16's 8 bits fit fp16's 11, and what is 2^-28 of the largest
// or less is rounded.  The weights p s are scaled likewise by the largest
// step and rounded to 11 bits.  (Two e4m3 terms per value, whose bytes 0000nnnn
// need even less unpacking, are no use: mma.sync has no fp8 path here, it is
// expanded into conversions and fp16 products, 24 to 37 cycles instead of 8.)
//
// fp32: queries and weights are split into three bf16 terms (24 bits); codes
// become 16 + n, exact in bf16, by dropping four bits into the mantissa of
// 16.0, then n - 7.5 by one subtraction, so that sums stay short.
//
// Bound: HBM (144 bytes per position and key/value head at head_dim 128) in
// principle; in fact nothing is full (HBM 64% of the copy rate, issue slots and
// integer pipe 58%): the 16 warps of an SM, all that 128 registers a thread
// leave room for, do not cover the fixed latencies of the 660 instructions that
// a unit takes a warp at head_dim 128.  32 sequences x 40 heads x up to 2304
// positions: 77 us, 4.2 TB/s (the bytes alone: 49 us);
// 131071 positions, 64 heads on 8: 46 us (23 us), 8 of them the join.  With
// codes turned into bf16 16 + n by three instructions per operand instead of
// one mask the former took 109 us.  A query column is one (token, head) of a
// key/value head's group; 8 columns cost what one costs.  Decoding has too few
// columns for tcgen05 (M = 128).
//
// Split: a unit is 32 positions of one (sequence, key/value head, column
// tile), a single 4608-byte bulk copy.  All units of the call are cut into
// equal contiguous ranges, one per CTA and in it one per warp; lengths are
// read on the device, so the launch depends on none of them.  A warp streams
// its range through a ring of its own, without meeting the others, and keeps
// a running maximum and sum per column.  What begins and ends inside its
// range it writes out; the parts of a pair that spans warps are joined in
// shared memory, and those of a pair that spans CTAs go to the workspace,
// where a second kernel joins them, always in the order of the positions.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "tcgen05.cuh"

#include <algorithm>
#include <type_traits>

namespace {

using namespace tc;

constexpr int WARPS = 8;
constexpr int STAGES = 2;        // 16 warps x 2 units in flight per SM: 147 KB, three times what the latency needs
constexpr int THREADS = WARPS * 32;
constexpr int MAX_B = LLAMA_PLAN_MAX_BATCH;

// What the second kernel joins at a CTA: the pair that begins in it and goes
// on in the `more` CTAs after it (0: none)
struct Join {
    int more, row0, head, col0, n_cols, pad[3];
};

// The sequences, and the units of the sequences 0 .. b, into shared memory
template <int COLS>
__device__ __forceinline__ long long unit_ends(const AttnArgs& a, Seq* seqs, long long* ends, long long* part) {
    const int beyond = a.split ? columns_beyond<WARPS>(a, seqs, ends, part) : 0;
    return prefix<WARPS>(a.B, ends, part, [&](int b) {
        Seq s = a.split ? seqs[b] : read_seq(a, b);
        if (a.split && many_columns(a, s, beyond)) s.n = 0;       // the other kernel's
        seqs[b] = s;
        return (long long)s.tiles<COLS>(a.G) * s.blocks() * a.n_kv;
    });
}

// Ranges: CTA c of C has units [U c / C, U (c + 1) / C); C <= U, so none is
// empty.  One unit per warp at least, before another CTA is used.
__device__ __forceinline__ long long range_start(long long U, int C, int c) { return U * c / C; }
__device__ __forceinline__ int cta_of_unit(long long U, int C, long long u) { return (int)(((u + 1) * C + U - 1) / U) - 1; }
__device__ __forceinline__ int live_ctas(long long U, int grid) {
    const long long c = (U + WARPS - 1) / WARPS;
    return (int)(c < grid ? c : grid);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Codes i and i + 4 of a word as bf16 16 + n, in the low and high half: the
// code goes to mantissa bits 3..6.  `mask` is 0x00780078 in a register that
// the compiler does not know: a logic operation takes one constant only.
__device__ __forceinline__ uint32_t codes16(uint32_t w, int i, uint32_t mask) {   // i known at compile time
    return ((i == 0 ? w << 3 : w >> (4 * i - 3)) & mask) | 0x41804180u;
}
// 16 + n less 23.5: n - 7.5, exactly
__device__ __forceinline__ uint32_t centred(uint32_t w) {
    __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&w);
    v = __hsub2(v, __floats2bfloat162_rn(23.5f, 23.5f));
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// (x, y) as SPL bf16 pairs whose sum is the pair (24 bits for SPL = 3); t[] low half = x
template <int SPL>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[SPL]) {
    t[0] = pack_bf16x2(x, y);
#pragma unroll
    for (int i = 1; i < SPL; ++i) {
        x -= lo_bf16(t[i - 1]);
        y -= hi_bf16(t[i - 1]);
        t[i] = pack_bf16x2(x, y);
    }
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// Bounded wait of a whole warp (all lanes poll); false after the limit
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer();
    while (!mbar_try_wait(bar, parity))
        if (global_timer() - t0 > WAIT_LIMIT_NS) return false;
    return true;
}

// 8 consecutive channels of a query row as bf16 pairs (i, i + 4), i = 0..3, in
// SPL terms; and their sum
template <int SPL>
__device__ __forceinline__ float load_pairs(const float* p, uint32_t (&r)[4][SPL]) {
    const float4 a = *(reinterpret_cast<const float4*>(p)), b = *(reinterpret_cast<const float4*>(p) + 1);
    split2<SPL>(a.x, b.x, r[0]);
    split2<SPL>(a.y, b.y, r[1]);
    split2<SPL>(a.z, b.z, r[2]);
    split2<SPL>(a.w, b.w, r[3]);
    return ((a.x + b.x) + (a.y + b.y)) + ((a.z + b.z) + (a.w + b.w));
}

__device__ __forceinline__ void put8(bf16* p, const float (&y)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}
__device__ __forceinline__ void put8(float* p, const float (&y)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}

// A unit's place, and (for the copy) its source
struct Unit {
    int b, head, tile, blk;     // sequence, key/value head, column tile, block of 32 positions
    const uint8_t* src;         // NULL: nothing to read
};

template <int HD, int NT>
struct Cfg {
    static constexpr int PART = HD + 4;          // floats of a part's column: output, maximum, sum, padding
    static constexpr int COLS = 8 * NT;
    static constexpr int BYTES = kv4::blk_bytes(HD);
    static constexpr int RING = WARPS * STAGES * BYTES;
    // ring (a warp's last part takes the place of its stages), scan, barriers, a first part per warp, unit ends,
    // sequences
    static constexpr int smem(int cols, int B) {
        return RING + WARPS * 8 + WARPS * STAGES * 8 + WARPS * cols * PART * 4 + B * (8 + (int)sizeof(Seq));
    }
    static_assert(STAGES * BYTES >= COLS * PART * 4, "a part fits the ring");
};

// Adds parts in order: weights 2^(m - M) of each, output and sum in fp32
template <int PER>
struct Sum {
    float y[PER] = {}, L = 0.f;
    __device__ __forceinline__ void add(const float (&x)[PER], float mw, float lw, float M) {
        // a part without a maximum holds nothing, or a NaN
        const float f = mw == -INFINITY ? (lw == 0.f ? 0.f : 1.f) : ex2(mw - M);
        L = fmaf(lw, f, L);
#pragma unroll
        for (int i = 0; i < PER; ++i) y[i] = fmaf(x[i], f, y[i]);
    }
};
template <int PER>
__device__ __forceinline__ void get(const float* p, float (&x)[PER]) {   // PER neighbouring floats
    if constexpr (PER == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2*>(p);
        x[0] = v.x; x[1] = v.y;
    }
}
__device__ __forceinline__ void put(bf16* p, const float (&y)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}
__device__ __forceinline__ void put(bf16* p, const float (&y)[2]) { *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(y[0], y[1]); }
__device__ __forceinline__ void put(float* p, const float (&y)[4]) { *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]); }
__device__ __forceinline__ void put(float* p, const float (&y)[2]) { *reinterpret_cast<float2*>(p) = make_float2(y[0], y[1]); }
// What a unit's arithmetic has to know of its pair
struct Pair {
    Seq sq;
    int head, tile;
    int first_pos;              // position of the sequence's first new token
    int fewest;                 // position of the tile's first token, which sees the fewest
};

// Shared by both cores: where column `col` of a pair's tile is written
template <typename T, int HD>
__device__ __forceinline__ T* out_row(const AttnArgs& a, const Pair& p, int gc) {
    return static_cast<T*>(a.o) + (int64_t)(p.sq.row0 + gc / a.G) * ((int64_t)a.H * HD) + (p.head * a.G + gc % a.G) * HD;
}
template <typename T, int HD>
__device__ __forceinline__ const T* query_row(const AttnArgs& a, const Pair& p, int gc) {   // column 0's for a column that is not there
    if (gc >= p.sq.n * a.G) gc = 0;
    return static_cast<const T*>(a.q) + (int64_t)(p.sq.row0 + gc / a.G) * a.q_stride + (p.head * a.G + gc % a.G) * HD;
}
// z and s of a row's groups
template <int GR>
__device__ __forceinline__ void scale_words(const uint8_t* p, int key, uint32_t (&y)[GR]) {
    if constexpr (GR == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p + key * 8);
        y[0] = v.x;
        y[1] = v.y;
    } else {
        y[0] = *reinterpret_cast<const uint32_t*>(p + key * 4);
    }
}

// ------------------------------------------------------------- bf16 core
// mma.m16n8k16 fp16: rows are keys, columns queries.  A lane has the columns
// 2 t, 2 t + 1 and, of a unit's 32 keys, the four 16 kb + 8 h + pi.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// A word's codes i and i + 4 as fp16 pairs: f[0] (i = 0) and f[2] (i = 2) n 2^-24,
// f[1] (i = 1) and f[3] (i = 3) 16 n 2^-24
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&f)[4]) {
    const uint32_t h = w >> 8;
    f[0] = w & 0x000f000fu;
    f[1] = w & 0x00f000f0u;
    f[2] = h & 0x000f000fu;
    f[3] = h & 0x00f000f0u;
}

template <int HD, int NT>
struct CoreBf16 {
    using T = bf16;
    static constexpr int COLS = 8 * NT, GR = kv4::groups(HD), PART = HD + 4, WPL = GR * 2, CTAS = NT == 1 ? 2 : 1;
    uint32_t q[NT][WPL][4];     // per word of codes: pairs (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16
    float qa[NT][2], qs[NT][2][GR];   // columns 2 t, 2 t + 1: base-2 scores per unit of the products, sums of q in those units
    float acc[NT][GR][4][4];    // [.][channel pair][row, col as mma's d]; odd channels 16-fold
    float m[NT][2], l[NT][2], zs[NT][2][GR];      // maximum, sum of weights, sum of weights times z
    float minus[NT][2];         // what scores are shifted by: minus the maximum, 0 before there is one
    uint32_t limit[GR];         // steps from here on (as bits, in the scale word) need another factor
    // what steps are multiplied with for fp16, a power of two: the largest a column saw comes to 2^5 .. 2^6 (the same
    // for all columns until one of several tokens is cut off; those units come last).  Biased exponents, byte
    // 2 c + gr of a column tile's word; 0: none yet
    uint32_t fits[NT];
    int g, t, pi, k2, k3;

    __device__ __forceinline__ uint32_t fit_exponent(int nt, int c, int gr) const { return __byte_perm(fits[nt], 0, 0x4440 | (2 * c + gr)); }
    __device__ __forceinline__ float fit(int nt, int c, int gr) const { return __uint_as_float(fit_exponent(nt, c, gr) << 23); }

    __device__ __forceinline__ explicit CoreBf16(int lane)
        : g(lane >> 2), t(lane & 3), pi(g ^ ((g >> 1) & 1)), k2((2 * t) ^ (t & 1)), k3((2 * t + 1) ^ (t & 1)) {}

    __device__ __forceinline__ void begin(const AttnArgs& a, const Pair& p) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int gc = p.tile * COLS + nt * 8 + g;      // this lane's column of the query operand
            const bf16* row = query_row<bf16, HD>(a, p, gc);
            uint4 raw[WPL];
#pragma unroll
            for (int wd = 0; wd < WPL; ++wd)      // word wd: piece 2 t + wd / GR, group wd % GR
                raw[wd] = gc < p.sq.n * a.G
                              ? *(reinterpret_cast<const uint4*>(row + (wd % GR) * kv4::GROUP + 8 * (2 * t + wd / GR)))
                              : make_uint4(0, 0, 0, 0);
            float top = 0.f, sum[GR];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) sum[gr] = 0.f;
#pragma unroll
            for (int wd = 0; wd < WPL; ++wd) {
                const uint32_t u[4] = {raw[wd].x, raw[wd].y, raw[wd].z, raw[wd].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = lo_bf16(u[i]), y = hi_bf16(u[i]);
                    top = max_nan(top, max_nan(fabsf(x), fabsf(y)));
                    sum[wd % GR] += x + y;
                }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], o);
            }
            const int e = (int)(__float_as_uint(top) >> 23);              // the exponent (biased), 255 for inf and NaN
            const int ec = min(max(e, 40), 240);
            const float up = __uint_as_float((uint32_t)(268 - ec) << 23);  // 2^14 for 2^(ec - 127)
            // true q . n = 2^24 / up of the product's: 2^(ec - 117)
            const float a_scale = a.scale * __uint_as_float((uint32_t)(ec + 10) << 23);
            // 2^(117 - ec); a query that is not finite makes its scores NaN, not the scale that hidden keys' -inf meet too
            const float unit = e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(244 - ec) << 23);
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                sum[gr] *= unit;
                qs[nt][0][gr] = __shfl_sync(0xffffffffu, sum[gr], 8 * t);
                qs[nt][1][gr] = __shfl_sync(0xffffffffu, sum[gr], 8 * t + 4);
            }
            qa[nt][0] = __shfl_sync(0xffffffffu, a_scale, 8 * t);
            qa[nt][1] = __shfl_sync(0xffffffffu, a_scale, 8 * t + 4);
#pragma unroll
            for (int wd = 0; wd < WPL; ++wd) {
                const uint32_t u[4] = {raw[wd].x, raw[wd].y, raw[wd].z, raw[wd].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {     // channels i and i + 4
                    const float f = i & 1 ? up * 0.0625f : up;
                    const float x = (i & 1 ? hi_bf16(u[i / 2]) : lo_bf16(u[i / 2])) * f;
                    const float y = (i & 1 ? hi_bf16(u[2 + i / 2]) : lo_bf16(u[2 + i / 2])) * f;
                    q[nt][wd][i] = pack_f16x2(x, y);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[nt][c] = -INFINITY;
                minus[nt][c] = 0.f;
                l[nt][c] = 0.f;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) zs[nt][c][gr] = 0.f;
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) acc[nt][gr][x][y] = 0.f;
        }
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) limit[gr] = 0;       // the first unit sets it
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) fits[nt] = 0;
    }

    // One unit from shared memory.  CUT: some (key, column) of it is hidden.
    template <bool CUT>
    __device__ __forceinline__ void unit(const AttnArgs& a, const Pair& pr, const uint8_t* kc, int key0) {
        const uint8_t* kp = kc + kv4::BLK * HD / 2;
        const uint8_t* vc = kc + kv4::half_bytes(HD);
        const uint8_t* vp = vc + kv4::BLK * HD / 2;
        // scores of 32 keys: sc[nt][key block][row half][column]
        float sc[NT][2][2][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint32_t wk[2][WPL];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* row = kc + (16 * kb + 8 * h + pi) * (HD / 2);
                if constexpr (GR == 2) {
                    const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * t);
                    wk[h][0] = x.x; wk[h][1] = x.y; wk[h][2] = x.z; wk[h][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(row + 8 * t);
                    wk[h][0] = x.x; wk[h][1] = x.y;
                }
            }
            float d[NT][GR][4];
#pragma unroll
            for (int wd = 0; wd < WPL; ++wd) {
                uint32_t f[2][4];
                codes_f16(wk[0][wd], f[0]);
                codes_f16(wk[1][wd], f[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x[4] = {f[0][2 * h], f[1][2 * h], f[0][2 * h + 1], f[1][2 * h + 1]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (wd < GR && h == 0) mma_f16_new(d[nt][wd % GR], x, q[nt][wd][0], q[nt][wd][1]);
                        else mma_f16(d[nt][wd % GR], x, q[nt][wd][2 * h], q[nt][wd][2 * h + 1]);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = 16 * kb + 8 * h + pi;
                uint32_t y[GR];
                scale_words<GR>(kp, key, y);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = 0.f;
#pragma unroll
                        for (int gr = 0; gr < GR; ++gr) {
                            v = gr == 0 ? hi_bf16(y[gr]) * d[nt][gr][2 * h + c] : fmaf(hi_bf16(y[gr]), d[nt][gr][2 * h + c], v);
                            v = fmaf(lo_bf16(y[gr]), qs[nt][c][gr], v);
                        }
                        if constexpr (CUT) {      // a column sees the keys up to its token's position
                            if (key0 + key > pr.first_pos + (pr.tile * COLS + nt * 8 + 2 * t + c) / a.G || key0 + key >= pr.sq.len) v = -INFINITY;
                        }
                        sc[nt][kb][h][c] = v;
                    }
            }
        }
        // the values' scales; what no column sees may be anything
        uint32_t y[2][2][GR];
        bool move = false;
        const int most = CUT ? pr.first_pos + min((pr.tile * COLS + COLS - 1) / a.G, pr.sq.n - 1) : 0;   // the tile's last token
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = 16 * kb + 8 * h + pi;
                scale_words<GR>(vp, key, y[kb][h]);
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    if (CUT && key0 + key > most) y[kb][h][gr] = 0;
                    move |= y[kb][h][gr] >= limit[gr];
                }
            }
        // running maximum: moved only when a column's scores pass it by more
        // than 8 (the weights stay below 2^8), so the sums are rescaled rarely
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = fmaxf(fmaxf(sc[nt][0][0][c], sc[nt][0][1][c]), fmaxf(sc[nt][1][0][c], sc[nt][1][1][c])) * qa[nt][c];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
                mx[nt][c] = v;
                move |= v > m[nt][c] + 8.f;       // -inf + 8 = -inf: the first score moves it
            }
        if (__any_sync(0xffffffffu, move)) {
            if (CUT && pr.fewest != most) rescale<true>(y, sc, mx);
            else rescale<false>(y, sc, mx);       // all columns see the same
        }
        // weights, and the weighted values
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint32_t p[NT][GR][2];                // weights times step: [key half]: rows keys, columns 2 t, 2 t + 1
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float s[GR], z[GR];
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    s[gr] = CUT ? hi_bf16(y[kb][h][gr]) : hi_bf16(y[kb][h][gr]) * fit(0, 0, gr);
                    z[gr] = lo_bf16(y[kb][h][gr]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float e[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        e[c] = ex2(fmaf(sc[nt][kb][h][c], qa[nt][c], minus[nt][c]));
                        l[nt][c] += e[c];
                    }
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) {
                        float w[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            // a key that this column does not see weighs nothing, also where its step is NaN
                            const bool none = CUT && sc[nt][kb][h][c] == -INFINITY;
                            w[c] = none ? 0.f : e[c] * (CUT ? s[gr] * fit(nt, c, gr) : s[gr]);
                            zs[nt][c][gr] = none ? zs[nt][c][gr] : fmaf(e[c], z[gr], zs[nt][c][gr]);
                        }
                        p[nt][gr][h] = transpose8x8(pack_f16x2(w[0], w[1]));
                    }
                }
            }
            uint32_t wv[4][GR];                   // piece g of the keys at k positions 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = 16 * kb + (x & 2) * 4 + ((x & 1) ? k3 : k2);
                if constexpr (GR == 2) {
                    const uint2 v = *reinterpret_cast<const uint2*>(vc + key * (HD / 2) + 8 * g);
                    wv[x][0] = v.x;
                    wv[x][1] = v.y;
                } else {
                    wv[x][0] = *reinterpret_cast<const uint32_t*>(vc + key * (HD / 2) + 4 * g);
                }
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int hw = 0; hw < 2; ++hw) {  // low and high four channels of the word
                    uint32_t f[2][4];             // [keys 2 t, 2 t + 1, or 8 on][channel]
                    codes_f16(__byte_perm(wv[0][gr], wv[1][gr], hw ? 0x7632 : 0x5410), f[0]);
                    codes_f16(__byte_perm(wv[2][gr], wv[3][gr], hw ? 0x7632 : 0x5410), f[1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t v[4] = {f[0][2 * x], f[0][2 * x + 1], f[1][2 * x], f[1][2 * x + 1]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][gr][hw * 2 + x], v, p[nt][gr][0], p[nt][gr][1]);
                    }
                }
        }
    }

    // New maxima and, where a step that a column sees passed what its factor allows for, a new factor.  What a
    // column does not see does not count: next to a step 2^20 times as large its own would be rounded away.
    template <bool APART>
    __device__ __forceinline__ void rescale(const uint32_t (&y)[2][2][GR], const float (&sc)[NT][2][2][2], const float (&mx)[NT][2]) {
        float more[NT][2][GR];
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
            uint32_t least = ~0u;
#pragma unroll
            for (int nt = 0; nt < (APART ? NT : 1); ++nt)
#pragma unroll
                for (int c = 0; c < (APART ? 2 : 1); ++c) {
                    uint32_t top = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t v = y[x / 2][x % 2][gr];
                        const bool out = v >= 0x7f800000u || (APART && sc[nt][x / 2][x % 2][c] == -INFINITY);     // NaN, or not seen
                        top = max(top, out ? 0u : v);
                    }
                    if constexpr (APART) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    } else {
                        top = __reduce_max_sync(0xffffffffu, top);
                    }
                    const uint32_t now = fit_exponent(nt, c, gr);
                    uint32_t lim = now == 0 ? 0u : (260u - now) << 23;                    // the step that passes it
                    float x = 1.f;
                    if (top >= lim) {
                        const uint32_t e = min(max(top >> 23, 8u), 250u), f = 259u - e;   // 2^5 for 2^(e - 127)
                        if (now != 0) x = ex2((float)((int)f - (int)now));                // nothing is summed before the first
                        fits[nt] += (f - now) * (APART ? 1u << (8 * (2 * c + gr)) : 0x00010001u << (8 * gr));
                        if constexpr (!APART)
#pragma unroll
                            for (int k = 1; k < NT; ++k) fits[k] = fits[0];
                        lim = (e + 1) << 23;
                    }
#pragma unroll
                    for (int k = 0; k < 2 * NT; ++k)
                        if (!APART || (k == 2 * nt + c)) more[k / 2][k % 2][gr] = x;
                    least = min(least, lim);
                }
            limit[gr] = APART ? __reduce_min_sync(0xffffffffu, least) : least;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float nm = fmaxf(m[nt][c], mx[nt][c]);
                const float f = nm == -INFINITY ? 1.f : ex2(m[nt][c] - nm);
                m[nt][c] = nm;
                minus[nt][c] = nm == -INFINITY ? 0.f : -nm;
                l[nt][c] *= f;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    zs[nt][c][gr] *= f;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        acc[nt][gr][x][c] *= f * more[nt][c][gr];
                        acc[nt][gr][x][2 + c] *= f * more[nt][c][gr];
                    }
                }
            }
    }

    // Ends the columns' sums: to the output if the range holds all of the pair, else to `dst` as a part
    __device__ __forceinline__ void finish(const AttnArgs& a, const Pair& p, bool whole, float* dst) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {        // over the lanes that share columns
                    l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], o);
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) zs[nt][c][gr] += __shfl_xor_sync(0xffffffffu, zs[nt][c][gr], o);
                }
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = nt * 8 + 2 * t + c, gc = p.tile * COLS + col;
                if (gc >= p.sq.n * a.G) continue;
                const float inv = whole ? inverse(l[nt][c]) : 1.f;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const float unfit = __uint_as_float((254u - fit_exponent(nt, c, gr)) << 23);      // nothing summed yet: 0 times it
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[2 * i] = fmaf(acc[nt][gr][i][c] * 16777216.f, unfit, zs[nt][c][gr]) * inv;
                        y[2 * i + 1] = fmaf(acc[nt][gr][i][2 + c] * 1048576.f, unfit, zs[nt][c][gr]) * inv;
                    }
                    const int ch = gr * kv4::GROUP + 8 * g;
                    if (whole) put8(out_row<bf16, HD>(a, p, gc) + ch, y);
                    else put8(dst + col * PART + ch, y);
                }
                if (!whole && g == 0) {
                    dst[col * PART + HD] = m[nt][c];
                    dst[col * PART + HD + 1] = l[nt][c];
                }
            }
    }
};

// ------------------------------------------------------------- fp32 core
// mma.m16n8k16 bf16: rows are keys, columns queries.  A lane has the columns
// 2 t, 2 t + 1 and, of a unit's 32 keys, the four 16 kb + 8 h + pi.
template <int HD, int NT>
struct CoreF32 {
    using T = float;
    static constexpr int COLS = 8 * NT, GR = kv4::groups(HD), PART = HD + 4, WPL = GR * 2, CTAS = 1, SPL = 3;
    uint32_t q[NT][WPL * 2][2][SPL];              // [column tile][word pair k-step][b0, b1][term]
    float qs[NT][2][GR];                          // sums of q over a group, columns 2 t, 2 t + 1
    float acc[NT][GR][4][4];                      // [.][channel pair][row, col as mma's d]
    float m[NT][2], l[NT][2], zs[NT][2][GR];      // maximum, sum of weights, sum of weights times (z + 7.5 s)
    int g, t, pi, k2, k3;
    uint32_t mask;

    // One 16-deep step, smallest terms first; sums over steps are fp32 additions: the tensor cores' do not round to
    // nearest, which shows in the sixth digit (12 heads over 6000 positions: 2.5e-6 of a head's norm, like this 7e-7)
    __device__ __forceinline__ static void product(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b0)[SPL], const uint32_t (&b1)[SPL]) {
        mma_bf16_new(d, a[0], a[1], a[2], a[3], b0[SPL - 1], b1[SPL - 1]);
#pragma unroll
        for (int x = SPL - 2; x >= 0; --x) mma_bf16(d, a[0], a[1], a[2], a[3], b0[x], b1[x]);
    }

    __device__ __forceinline__ explicit CoreF32(int lane)
        : g(lane >> 2), t(lane & 3), pi(g ^ ((g >> 1) & 1)), k2((2 * t) ^ (t & 1)), k3((2 * t + 1) ^ (t & 1)) {
        asm volatile("mov.b32 %0, 0x00780078;" : "=r"(mask));
    }

    __device__ __forceinline__ void begin(const AttnArgs& a, const Pair& p) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int gc = p.tile * COLS + nt * 8 + g;      // this lane's column of the query operand
            const bool on = gc < p.sq.n * a.G;
            const float* qp = query_row<float, HD>(a, p, gc);
            float sum[GR];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) sum[gr] = 0.f;
#pragma unroll
            for (int wd = 0; wd < WPL; ++wd) {            // word wd: piece 2 t + wd / GR, group wd % GR
                uint32_t r[4][SPL];
                const float s = load_pairs<SPL>(qp + (wd % GR) * kv4::GROUP + 8 * (2 * t + wd / GR), r);
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int x = 0; x < SPL; ++x) q[nt][wd * 2 + h / 2][h & 1][x] = on ? r[h][x] : 0u;
                sum[wd % GR] += on ? s : 0.f;
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
                sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
                qs[nt][0][gr] = __shfl_sync(0xffffffffu, sum[gr], 8 * t);
                qs[nt][1][gr] = __shfl_sync(0xffffffffu, sum[gr], 8 * t + 4);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[nt][c] = -INFINITY;
                l[nt][c] = 0.f;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) zs[nt][c][gr] = 0.f;
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[nt][gr][x][y] = 0.f;
                }
        }
    }

    // One unit from shared memory.  CUT: some (key, column) of it is hidden.
    template <bool CUT>
    __device__ __forceinline__ void unit(const AttnArgs& a, const Pair& pr, const uint8_t* kc, int key0) {
        const uint8_t* kp = kc + kv4::BLK * HD / 2;
        const uint8_t* vc = kc + kv4::half_bytes(HD);
        const uint8_t* vp = vc + kv4::BLK * HD / 2;
        auto scales = [&](const uint8_t* p, int key, float (&z)[GR], float (&s)[GR]) {
            uint32_t y[GR];
            scale_words<GR>(p, key, y);
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                z[gr] = lo_bf16(y[gr]);
                s[gr] = hi_bf16(y[gr]);
            }
        };
        // scores of 32 keys: sc[nt][key block][row half][column]
        float sc[NT][2][2][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint32_t wk[2][WPL];
            float s[2][GR], z[2][GR];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = 16 * kb + 8 * h + pi;
                if constexpr (GR == 2) {
                    const uint4 x = *reinterpret_cast<const uint4*>(kc + key * (HD / 2) + 16 * t);
                    wk[h][0] = x.x; wk[h][1] = x.y; wk[h][2] = x.z; wk[h][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(kc + key * (HD / 2) + 8 * t);
                    wk[h][0] = x.x; wk[h][1] = x.y;
                }
                scales(kp, key, z[h], s[h]);
            }
            float d[NT][GR][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                    for (int x = 0; x < 4; ++x) d[nt][gr][x] = 0.f;
#pragma unroll
            for (int wd = 0; wd < WPL; ++wd)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        f[x] = codes16(wk[x & 1][wd], 2 * h + (x >> 1), mask);
                        f[x] = centred(f[x]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float part[4];
                        product(part, f, q[nt][wd * 2 + h][0], q[nt][wd * 2 + h][1]);
#pragma unroll
                        for (int x = 0; x < 4; ++x) d[nt][wd % GR][x] += part[x];
                    }
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float off[GR];
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) off[gr] = fmaf(7.5f, s[h][gr], z[h][gr]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = 0.f;
#pragma unroll
                        for (int gr = 0; gr < GR; ++gr) {
                            v = gr == 0 ? s[h][gr] * d[nt][gr][2 * h + c] : fmaf(s[h][gr], d[nt][gr][2 * h + c], v);
                            v = fmaf(off[gr], qs[nt][c][gr], v);
                        }
                        if constexpr (CUT) {      // a column sees the keys up to its token's position
                            const int key = key0 + 16 * kb + 8 * h + pi;
                            if (key > pr.first_pos + (pr.tile * COLS + nt * 8 + 2 * t + c) / a.G || key >= pr.sq.len) v = -INFINITY;
                        }
                        sc[nt][kb][h][c] = v;
                    }
            }
        }
        // running maximum: moved only when a column's scores pass it by more
        // than 8 (the weights stay below 2^8), so the sums are rescaled rarely
        bool move = false;
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = fmaxf(fmaxf(sc[nt][0][0][c], sc[nt][0][1][c]), fmaxf(sc[nt][1][0][c], sc[nt][1][1][c])) * a.scale;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
                mx[nt][c] = v;
                move |= v > m[nt][c] + 8.f;       // -inf + 8 = -inf: the first score moves it
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float nm = fmaxf(m[nt][c], mx[nt][c]);
                    const float f = nm == -INFINITY ? 1.f : ex2(m[nt][c] - nm);
                    m[nt][c] = nm;
                    l[nt][c] *= f;
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) {
                        zs[nt][c][gr] *= f;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            acc[nt][gr][x][c] *= f;
                            acc[nt][gr][x][2 + c] *= f;
                        }
                    }
                }
        }
        // weights, and the weighted values
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint32_t p[NT][GR][2][SPL];           // weights times step, rounded: [key half]: rows keys, columns 2 t, 2 t + 1
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = 16 * kb + 8 * h + pi;
                float s[GR], z[GR];
                scales(vp, key, z, s);
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    z[gr] = fmaf(7.5f, s[gr], z[gr]);
                    if (CUT && key0 + key >= pr.sq.len) z[gr] = s[gr] = 0.f;     // what lies behind the sequence may be anything
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float e[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        e[c] = ex2(fmaf(sc[nt][kb][h][c], a.scale, m[nt][c] == -INFINITY ? 0.f : -m[nt][c]));
                        l[nt][c] += e[c];
                    }
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) {
                        float w[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            // a key that this column does not see weighs nothing, also where its step is NaN
                            // (one that it sees may weigh 0 too: then NaN is NaN)
                            const bool none = CUT && sc[nt][kb][h][c] == -INFINITY;
                            w[c] = none ? 0.f : e[c] * s[gr];
                            zs[nt][c][gr] = none ? zs[nt][c][gr] : fmaf(e[c], z[gr], zs[nt][c][gr]);
                        }
                        split2<SPL>(w[0], w[1], p[nt][gr][h]);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int x = 0; x < SPL; ++x) p[nt][gr][h][x] = transpose8x8(p[nt][gr][h][x]);
                }
            uint32_t wv[4][GR];                   // piece g of the keys at k positions 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = 16 * kb + (x & 2) * 4 + ((x & 1) ? k3 : k2);
                if constexpr (GR == 2) {
                    const uint2 y = *reinterpret_cast<const uint2*>(vc + key * (HD / 2) + 8 * g);
                    wv[x][0] = y.x;
                    wv[x][1] = y.y;
                } else {
                    wv[x][0] = *reinterpret_cast<const uint32_t*>(vc + key * (HD / 2) + 4 * g);
                }
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int hw = 0; hw < 2; ++hw) {  // low and high four channels of the word
                    const uint32_t pr[2] = {__byte_perm(wv[0][gr], wv[1][gr], hw ? 0x7632 : 0x5410),
                                            __byte_perm(wv[2][gr], wv[3][gr], hw ? 0x7632 : 0x5410)};
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t f[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            f[y] = codes16(pr[y >> 1], 2 * x + (y & 1), mask);
                            f[y] = centred(f[y]);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float part[4];
                            product(part, f, p[nt][gr][0], p[nt][gr][1]);
#pragma unroll
                            for (int y = 0; y < 4; ++y) acc[nt][gr][hw * 2 + x][y] += part[y];
                        }
                    }
                }
        }
    }

    __device__ __forceinline__ void finish(const AttnArgs& a, const Pair& p, bool whole, float* dst) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {        // over the lanes that share columns
                    l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], o);
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) zs[nt][c][gr] += __shfl_xor_sync(0xffffffffu, zs[nt][c][gr], o);
                }
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = nt * 8 + 2 * t + c, gc = p.tile * COLS + col;
                if (gc >= p.sq.n * a.G) continue;
                const float inv = whole ? inverse(l[nt][c]) : 1.f;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[2 * i] = (acc[nt][gr][i][c] + zs[nt][c][gr]) * inv;
                        y[2 * i + 1] = (acc[nt][gr][i][2 + c] + zs[nt][c][gr]) * inv;
                    }
                    const int ch = gr * kv4::GROUP + 8 * g;
                    if (whole) put8(out_row<float, HD>(a, p, gc) + ch, y);
                    else put8(dst + col * PART + ch, y);
                }
                if (!whole && g == 0) {
                    dst[col * PART + HD] = m[nt][c];
                    dst[col * PART + HD + 1] = l[nt][c];
                }
            }
    }
};

// ------------------------------------------------------------- the kernel

template <template <int, int> class CoreOf, int HD, int NT>
__global__ void __launch_bounds__(THREADS, CoreOf<HD, NT>::CTAS) kv4_attn_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<HD, NT>;
    using Core = CoreOf<HD, NT>;
    using T = typename Core::T;
    constexpr int COLS = C::COLS, PART = C::PART, PER = HD / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long part_id[2 * WARPS];      // first unit of the pair a part belongs to, -1: no part
    __shared__ int4 part_of[2 * WARPS];           // its sequence's row0, head, first column, columns
    __shared__ int part_blocks[2 * WARPS];        // units of the pair
    long long* scan = reinterpret_cast<long long*>(smem + C::RING);
    float* firsts = reinterpret_cast<float*>(scan + WARPS + WARPS * STAGES);
    long long* ends = reinterpret_cast<long long*>(firsts + WARPS * a.cols * PART);
    Seq* seqs = reinterpret_cast<Seq*>(ends + a.B);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(smem) + warp * STAGES * C::BYTES;
    uint8_t* ring_p = smem + warp * STAGES * C::BYTES;
    const uint32_t bars = smem_u32(scan + WARPS) + warp * STAGES * 8;
    Join* join = reinterpret_cast<Join*>(a.work + (size_t)gridDim.x * 2 * a.cols * PART) + blockIdx.x;
    pdl_launch_dependents();
    if (lane == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(bars + 8 * s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < 2 * WARPS) part_id[threadIdx.x] = -1;
    pdl_wait();
    const long long U = unit_ends<COLS>(a, seqs, ends, scan);     // its barriers publish the mbarriers too
    const int n_ctas = live_ctas(U, gridDim.x);
    if ((int)blockIdx.x >= n_ctas) {
        if (threadIdx.x == 0) join->more = 0;
        return;
    }
    const long long lo = range_start(U, n_ctas, blockIdx.x), hi = range_start(U, n_ctas, blockIdx.x + 1);
    const long long u0 = lo + (hi - lo) * warp / WARPS;
    const int n_units = (int)(lo + (hi - lo) * (warp + 1) / WARPS - u0);
    const uint64_t policy = l2_evict_first();

    // the units of this warp, 32 at a time, one per lane
    auto describe = [&](int i) {
        Unit x{0, 0, 0, 0, nullptr};
        if (i >= n_units) return x;
        const long long u = u0 + i;
        x.b = seq_of_unit(ends, a.B, u);
        const Seq s = seqs[x.b];
        const long long r = u - (x.b ? ends[x.b - 1] : 0);      // 2^31 and more in a long prompt of many heads
        const int tiles = s.tiles<COLS>(a.G), blocks = s.blocks();
        const int pair = r < 0x7fffffff ? (int)r / blocks : (int)(r / blocks);
        x.blk = (int)(r - (long long)pair * blocks);
        x.head = pair / tiles;
        x.tile = pair - x.head * tiles;
        // the tile's last column sees the most; blocks past it are not read
        const int last_tok = min((x.tile * COLS + COLS - 1) / a.G, s.n - 1);
        if (x.blk * kv4::BLK <= s.len - s.n + last_tok) {
            const int page = a.table[(int64_t)x.b * a.pps + x.blk / (kv4::PAGE / kv4::BLK)];
            if (page >= 0 && page < a.n_pages)
                x.src = a.pool + kv4::blk_offset(page, a.n_kv, x.head, x.blk * kv4::BLK, HD);
            else
                atomicOr(a.err, LLAMA_DEVERR_INPUT);      // its positions are left out
        }
        return x;
    };
    Unit mine = describe(lane), next = mine;      // of the batch being read, and of the one being copied
    int issued = 0;
    auto issue = [&]() {                          // the next unit's copy, if there is one
        if (issued >= n_units) return;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(next.src), issued & 31));
        if (src && lane == 0) {
            const int s = issued % STAGES;
            mbar_expect_tx(bars + 8 * s, C::BYTES);
            bulk_copy(ring + s * C::BYTES, src, C::BYTES, bars + 8 * s, policy);
        }
        if ((++issued & 31) == 0) next = describe(issued + lane);
    };
    for (int s = 0; s < STAGES; ++s) issue();

    if (threadIdx.x == THREADS - 1) {             // for the second kernel: does the last pair begin here and go on?
        Join j{};
        const int b = seq_of_unit(ends, a.B, hi - 1);
        const Seq s = seqs[b];
        const long long base = b ? ends[b - 1] : 0;
        const int pair = (int)((hi - 1 - base) / s.blocks()), tiles = s.tiles<COLS>(a.G);
        const long long p0 = base + (long long)pair * s.blocks();
        if (p0 >= lo && p0 + s.blocks() > hi) {
            j.more = cta_of_unit(U, n_ctas, p0 + s.blocks() - 1) - (int)blockIdx.x;
            j.row0 = s.row0;
            j.head = pair / tiles;
            j.col0 = (pair - j.head * tiles) * COLS;
            j.n_cols = min(s.n * a.G - j.col0, COLS);
        }
        *join = j;
    }

    Core core(lane);
    Pair pr{{0, 0, 0}, -1, -1, 0, 0};
    int b = -1, first_blk = 0;
    uint32_t phases = 0;
    bool dead = false;
    // ends a pair's sums: whole if this warp has all of it, else a part in `slot`
    auto finish = [&](bool whole, int slot, float* dst, long long id) {
        core.finish(a, pr, whole, dst);
        if (!whole && lane == 0) {
            part_id[slot] = id;
            part_of[slot] = make_int4(pr.sq.row0, pr.head, pr.tile * COLS, min(pr.sq.n * a.G - pr.tile * COLS, COLS));
            part_blocks[slot] = pr.sq.blocks();
        }
    };
    for (int i = 0; i < n_units; ++i) {
        if (dead && i >= issued) break;           // nothing of this warp's is in flight any more
        const int from = i & 31;
        const int at = __shfl_sync(0xffffffffu, mine.src ? mine.blk : ~mine.blk, from);   // ~: nothing to read
        const bool held = at >= 0;
        const int blk = held ? at : ~at;
        if (i == 0 || blk == 0) {                 // another pair
            const int ub = __shfl_sync(0xffffffffu, mine.b, from), uh = __shfl_sync(0xffffffffu, mine.head, from);
            const int ut = __shfl_sync(0xffffffffu, mine.tile, from);
            // the pair before ended with its last unit: it is this warp's alone if it began here, else its end
            if (b >= 0) finish(first_blk == 0, 2 * warp, firsts + warp * a.cols * PART, u0 + i - pr.sq.blocks());
            b = ub;
            pr.sq = seqs[b];
            pr.head = uh;
            pr.tile = ut;
            pr.first_pos = pr.sq.len - pr.sq.n;
            pr.fewest = pr.first_pos + pr.tile * COLS / a.G;
            first_blk = blk;
            if (pr.sq.len == 0) {                 // nothing to see: zeros, and no pair is open
                const int cols = min(pr.sq.n * a.G - pr.tile * COLS, COLS);
                for (int e = lane; e < cols * (HD / PER); e += 32) {
                    const float zero[PER] = {};
                    put(out_row<T, HD>(a, pr, pr.tile * COLS + e / (HD / PER)) + e % (HD / PER) * PER, zero);
                }
                b = -1;
            } else {
                core.begin(a, pr);
            }
        }
        if (from == 31) mine = next;              // copies are ahead: their batch is the next one read
        if (!held) {
            if (!dead) issue();
            continue;
        }
        const int st = i % STAGES;
        if (!wait_bounded(bars + 8 * st, (phases >> st) & 1u)) {
            // the copy never landed: record it and look once more (bounded), so that it does not land in
            // the next CTA's shared memory; no further unit is issued or read
            if (lane == 0) atomicOr(a.err, LLAMA_DEVERR_TIMEOUT);
            wait_bounded(bars + 8 * st, (phases >> st) & 1u);
            dead = true;
        }
        phases ^= 1u << st;
        if (dead) continue;
        const int key0 = blk * kv4::BLK;
        if (key0 + kv4::BLK - 1 > pr.fewest || key0 + kv4::BLK > pr.sq.len)
            core.template unit<true>(a, pr, ring_p + st * C::BYTES, key0);
        else
            core.template unit<false>(a, pr, ring_p + st * C::BYTES, key0);
        __syncwarp();                             // every lane is done with the stage
        issue();
    }
    if (b >= 0) {
        const long long end = u0 + n_units, base = b ? ends[b - 1] : 0;
        const long long p0 = base + (end - 1 - base) / pr.sq.blocks() * pr.sq.blocks();
        finish(first_blk == 0 && end == p0 + pr.sq.blocks(), 2 * warp + 1, reinterpret_cast<float*>(ring_p), p0);
    }
    __syncthreads();

    // the parts of this CTA, joined pair by pair and column by column: lane k
    // looks at part k; a pair's parts follow one another
    const long long my_id = lane < 2 * WARPS ? part_id[lane] : -1;
    const unsigned there = __ballot_sync(0xffffffffu, my_id >= 0);
    const unsigned below = there & ((1u << lane) - 1u);
    const long long before = __shfl_sync(0xffffffffu, my_id, below ? 31 - __clz(below) : 0);
    unsigned firsts_of = __ballot_sync(0xffffffffu, my_id >= 0 && (!below || before != my_id));
    int item = 0;
    while (firsts_of) {
        const int j = __ffs(firsts_of) - 1;
        firsts_of &= firsts_of - 1;
        const unsigned run = there & ~((1u << j) - 1u) & (firsts_of ? (1u << (__ffs(firsts_of) - 1)) - 1u : ~0u);
        const long long id = part_id[j];
        const int4 of = part_of[j];
        const bool whole = id >= lo && id + part_blocks[j] <= hi;
        for (int col = 0; col < of.w; ++col, ++item) {
            if (item % WARPS != warp) continue;
            auto at = [&](int k) {
                return ((k & 1) ? reinterpret_cast<const float*>(smem + (k >> 1) * STAGES * C::BYTES) : firsts + (k >> 1) * a.cols * PART) +
                       col * PART;
            };
            const float M = warp_max((run >> lane) & 1u ? at(lane)[HD] : -INFINITY);
            Sum<PER> sum;
            for (unsigned r = run; r; r &= r - 1) {
                const float* part = at(__ffs(r) - 1);
                float x[PER];
                get<PER>(part + lane * PER, x);
                sum.add(x, part[HD], part[HD + 1], M);
            }
            if (whole) {
                const float inv = inverse(sum.L);
                const int gc = of.z + col;
                T* o = static_cast<T*>(a.o) + (int64_t)(of.x + gc / a.G) * ((int64_t)a.H * HD) + (of.y * a.G + gc % a.G) * HD;
#pragma unroll
                for (int i = 0; i < PER; ++i) sum.y[i] *= inv;
                put(o + lane * PER, sum.y);
            } else {
                float* w = a.work + (((size_t)blockIdx.x * 2 + (id >= lo ? 1 : 0)) * a.cols + col) * PART;
                put(w + lane * PER, sum.y);
                if (lane == 0) {
                    w[HD] = M;
                    w[HD + 1] = sum.L;
                }
            }
        }
    }
}

// Joins the parts of the pairs that span CTAs: CTA c takes the pair that
// begins in the first kernel's CTA c and goes on.  16 warps: as many per
// column as there are, each a stretch of the parts, eight in flight at once.
constexpr int JOIN_WARPS = 16;

template <typename T, int HD>
__global__ void __launch_bounds__(JOIN_WARPS * 32) kv4_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int PER = HD / 32, PART = HD + 4, DEEP = 8;
    __shared__ __align__(16) float sm[JOIN_WARPS][PART];
    pdl_launch_dependents();
    pdl_wait();
    const Join j = reinterpret_cast<const Join*>(a.work + (size_t)gridDim.x * 2 * a.cols * PART)[blockIdx.x];
    if (j.more <= 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = j.n_cols == 1 ? 16 : j.n_cols == 2 ? 8 : j.n_cols <= 4 ? 4 : j.n_cols <= 8 ? 2 : 1;
    const int col = warp / team, member = warp % team, n = j.more + 1;
    const int k0 = n * member / team, k1 = n * (member + 1) / team;
    auto at = [&](int k) {                        // part k: the pair's beginning here, then the CTAs after
        return a.work + (((size_t)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * a.cols + col) * PART;
    };
    float M = -INFINITY;                          // of this warp's parts
    Sum<PER> sum;
    if (col < j.n_cols) {
        for (int k = k0; k < k1; k += DEEP) {
            float x[DEEP][PER], mw[DEEP], lw[DEEP];
#pragma unroll
            for (int d = 0; d < DEEP; ++d) {
                const float* p = at(min(k + d, k1 - 1));
                get<PER>(p + lane * PER, x[d]);
                mw[d] = p[HD];
                lw[d] = p[HD + 1];
            }
            float nm = M;
#pragma unroll
            for (int d = 0; d < DEEP; ++d)
                if (k + d < k1) nm = fmaxf(nm, mw[d]);
            const float f = nm == -INFINITY ? 1.f : ex2(M - nm);
            M = nm;
            sum.L *= f;
#pragma unroll
            for (int i = 0; i < PER; ++i) sum.y[i] *= f;
#pragma unroll
            for (int d = 0; d < DEEP; ++d)
                if (k + d < k1) sum.add(x[d], mw[d], lw[d], M);
        }
    }
    put(&sm[warp][lane * PER], sum.y);
    if (lane == 0) {
        sm[warp][HD] = M;
        sm[warp][HD + 1] = sum.L;
    }
    __syncthreads();
    if (member > 0 || col >= j.n_cols) return;
    Sum<PER> all;
    float top = -INFINITY;
    for (int w = 0; w < team; ++w) top = fmaxf(top, sm[warp + w][HD]);
    for (int w = 0; w < team; ++w) {
        float x[PER];
        get<PER>(&sm[warp + w][lane * PER], x);
        all.add(x, sm[warp + w][HD], sm[warp + w][HD + 1], top);
    }
    const float inv = inverse(all.L);
#pragma unroll
    for (int i = 0; i < PER; ++i) all.y[i] *= inv;
    const int gc = j.col0 + col;
    put(static_cast<T*>(a.o) + (int64_t)(j.row0 + gc / a.G) * ((int64_t)a.H * HD) + (j.head * a.G + gc % a.G) * HD + lane * PER, all.y);
}

template <template <int, int> class CoreOf, int HD, int NT>
int run(AttnArgs& a, cudaStream_t st) {
    using C = Cfg<HD, NT>;
    using Core = CoreOf<HD, NT>;
    static PerDeviceOnce once;
    int rc = once_per_device(once, []() -> int {
        LLAMA_CUDA_TRY(cudaFuncSetAttribute(kv4_attn_kernel<CoreOf, HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            C::smem(C::COLS, MAX_B)));
        return (int)LLAMA_OK;
    });
    if (rc) return rc;
    const int ctas = std::min(tc_num_sms(), STEP_MAX_CTAS) * Core::CTAS;
    launch_pdl(kv4_attn_kernel<CoreOf, HD, NT>, dim3(ctas), dim3(THREADS), C::smem(a.cols, a.B), st, a);
    LLAMA_LAUNCH_CHECK();
    launch_pdl(kv4_join_kernel<typename Core::T, HD>, dim3(ctas), dim3(JOIN_WARPS * 32), 0, st, a);
    LLAMA_LAUNCH_CHECK();
    return LLAMA_OK;
}

// Column tiles of 16 once a sequence may bring more than 8 columns: the
// codes are then unpacked once for 16 (16 sequences x 2048 on 4 key/value
// heads of 128, 16 columns: 30.2 us, as two tiles of 8: 32.3).  Tiles of 16
// have one CTA per SM, so up to 8 columns those of 8 are faster (1 column,
// 32 x 32 heads x 2048: 73.9 against 98.7 us; 8 columns, 16 x 8 heads: 23.0
// against 24.2).
int col_tiles(int max_q, int G) { return (int64_t)max_q * G > 8 ? 2 : 1; }

}  // namespace

// Workspace: this kernel's parts, then those of the kernel of many columns
static uint64_t few_work_bytes(int G, int hd, int max_q) {
    const int nt = col_tiles(max_q, G);
    const int64_t cols = (int64_t)max_q * G < 8 * nt ? (int64_t)max_q * G : 8 * nt;
    return (uint64_t)2 * STEP_MAX_CTAS * (2 * cols * (hd + 4) * sizeof(float) + sizeof(Join));
}

uint64_t attention_kv4_work_bytes(int H, int n_kv, int hd, int max_q) {
    const int G = H / n_kv;
    return few_work_bytes(G, hd, max_q) + ((int64_t)max_q * G > TC_COLS ? attention_kv4_tc_work_bytes(hd) : 0);
}

int launch_attention_kv4(int dtype, const void* q, int64_t q_stride, const uint8_t* pool, int n_pages, const int32_t* table,
                         int pps, const int32_t* kv_len, const int32_t* cu, int max_q, void* o, int B, int rows, int H,
                         int n_kv, int hd, float* work, int* err, cudaStream_t st) {
    AttnArgs a;
    a.q = q;
    a.pool = pool;
    a.table = table;
    a.kv_len = kv_len;
    a.cu = cu;
    a.o = o;
    a.work = work;
    a.B = B;
    a.rows = rows;
    a.H = H;
    a.n_kv = n_kv;
    a.G = H / n_kv;
    a.pps = pps;
    a.n_pages = n_pages;
    a.max_q = max_q;
    a.q_stride = q_stride;
    const int nt = col_tiles(max_q, a.G);
    a.cols = (int64_t)max_q * a.G < 8 * nt ? max_q * a.G : 8 * nt;
    a.scale = 1.4426950408889634f / sqrtf((float)hd);
    a.split = dtype == LLAMA_BF16 && (int64_t)max_q * a.G > TC_COLS;
    a.tc_offset = few_work_bytes(a.G, hd, max_q);
    a.err = err;
    if (a.split) {
        const int rc = launch_attention_kv4_tc(&a, hd, st);
        if (rc) return rc;
    }
    if (dtype == LLAMA_BF16) {
        if (hd == 128) return nt == 1 ? run<CoreBf16, 128, 1>(a, st) : run<CoreBf16, 128, 2>(a, st);
        return nt == 1 ? run<CoreBf16, 64, 1>(a, st) : run<CoreBf16, 64, 2>(a, st);
    }
    if (hd == 128) return nt == 1 ? run<CoreF32, 128, 1>(a, st) : run<CoreF32, 128, 2>(a, st);
    return nt == 1 ? run<CoreF32, 64, 1>(a, st) : run<CoreF32, 64, 2>(a, st);
}
