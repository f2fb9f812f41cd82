// Attention of many new tokens (a prompt, or a chunk of one) over the 4-bit
// paged cache, on the tcgen05 tensor cores.
//
// A query column is a (token, head) pair of a key/value head's group; 128 of
// them fill a tile.  Per tile: O = softmax(Q K^T / sqrt(hd) + causal mask) V
// over the pages the tile's last token sees, with K = z + n s and V alike
// turned into fp16 tiles in shared memory as they are needed, so a page is
// unpacked once for 256 columns (two adjacent tiles of an item) instead of
// once for 16 as in the kernel for few columns (kv4_attn.cu).
//
// An item is two adjacent tiles of one sequence and key/value head; its pages
// are its units, and all units are cut into equal contiguous ranges, one per
// CTA (one per SM), so that a few items fill the SMs too.  Parts of items
// that span CTAs go to the workspace and are joined by a second kernel, in
// the order of the positions.
//
// Roles (14 warps):
//   warps 0, 1   MMA issuers of tiles 0 and 1 (warp 0 also has the tensor
//                memory): S = Q K_j^T -> TMEM, then O += P(j) V_j with P read
//                from TMEM (written over S by the softmax).  One thread
//                polling for both tiles took 1200 clocks to notice a P.
//   warps 2..5   softmax of tile 0, 6..9 of tile 1: a query column per
//                thread; they also bring the columns' queries to shared
//                memory and write the outputs.
//   warps 10..13 unpacking: a position per thread; its packed row of the
//                next page is on its way while this one is converted.
// Bound: the chain S -> softmax -> P V of a tile, 8000 clocks per page for both
// tiles (the special-function unit alone, one 2^x per score: 2048; products:
// about 3200), since P lies over S and the next S waits for P V.  Scores are
// read twice because 14 warps leave 128 registers a thread.  Unpacking (about
// 500 instructions per thread and page, 4 warps) hides beside it.  4 requests
// of 1381 .. 2176 positions with 448, 384, 512 and 1 new tokens, 32 heads on 8 of
// 128: 110 us, about 85 here and 15 in the join; one issuer polling for both
// tiles took 10 more.
//
// Numbers: keys, values, queries and weights are fp16 here (11 bits; bf16's 8
// cost twice the output's own rounding, 3.9e-3 instead of 1.7e-3 of it), so
// their ranges are looked after: a page's keys, and its values, are scaled by
// the power of two that brings the page's largest to 2^10 .. 2^11, a column's
// query likewise; scores are multiplied back in fp32, and the outputs so far
// are brought to the page's scale where that is more than 2^8 off (else the
// weights carry the difference).  A code becomes 1024 + n or
// 1024 + 16 n in fp16 (a mask and an or), n exactly by one operation, and
// z + n s by one fused multiply-add with one rounding.  Scores, maxima, sums
// and outputs are fp32.  The channels of 8 neighbours stand as c0 c4 c1 c5 c2
// c6 c3 c7, the order in which masks take them out of a word: the queries
// are stored in the same order, and the outputs are put back in theirs.
//
// Where some row's keys are 2^8 below the page's largest (outliers among
// them), every row has a factor of its own, which goes to the scores.  A key's
// channels share one: those 2^-24 of the key's largest and less are rounded
// away.  Where some 64 channels of a row's values are 2^8 below the page's
// largest, the page's values are bf16, unscaled, and its weights two bf16
// terms, relative to the largest values that the column sees: bf16 holds any
// size of them (their 8 bits are those of a bf16 cache).  With fp16 and a
// factor per row, 64 channels much smaller than the row's others were lost,
// and small values beside large ones of little weight.  So a column is not
// touched by the size of what it does not see, nor one half of a head by that
// of the other.
//
// A page outside the pool is not seen.  A group of values that holds NaN is
// unpacked as zeros and its positions noted, and a column that sees one of
// them gets NaN in that group: a position that a column does not see cannot
// reach it through 0 * NaN.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "tcgen05.cuh"

namespace {

using namespace tc;
using namespace kv4;

constexpr int BQ = 128;              // columns per tile
constexpr int BKV = PAGE;            // positions per key / value tile
constexpr int NTHREADS = 14 * 32;
constexpr int SOFT0 = 2, UNPACK0 = 10;
constexpr int NS = 2;                // stages of the key and value rings
constexpr int NF = 4;                // pages whose notes are kept
constexpr float RESCALE_LOG2 = 8.f;  // move the running maximum only by more than this
constexpr float LIFT = 128.f, LIFT_LOG2 = 7.f;     // weights as fp16 are lifted to the end of its range: 2^15, and 11 bits down to 2^-21
constexpr int ITEM = 2 * BQ;         // columns of an item

constexpr int B_QFULL = 0, B_QEMPTY = 8, B_KFULL = 16, B_KEMPTY = B_KFULL + 8 * NS, B_VFULL = B_KEMPTY + 8 * NS;
constexpr int B_VEMPTY = B_VFULL + 8 * NS, B_SFULL = B_VEMPTY + 8 * NS, B_PFULL = B_SFULL + 16, B_PVDONE = B_PFULL + 16;
constexpr int B_OLAST = B_PVDONE + 16, B_OFREE = B_OLAST + 16, B_DRAIN = B_OFREE + 16, B_TOPS = B_DRAIN + 16, B_END = B_TOPS + 8;

template <int HD>
struct TCfg {
    static constexpr int REG = 128 * 128;            // [128 rows][64 numbers of 16 bits], 128-byte swizzle
    static constexpr int NREG = HD / 64;
    static constexpr int TILE = NREG * REG;
    static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + NS * TILE, OFF_BAR = OFF_V + NS * TILE;
    static constexpr int OFF_NOTES = OFF_BAR + 256;  // TMEM slot and abort flag in the barriers' block
    static constexpr int OFF_ROWS = OFF_NOTES + NF * 64;     // factors of the rows of wide pages
    static constexpr int OFF_SCAN = OFF_ROWS + NF * 1024;    // scan, and the unpacking warps' maxima and minima
    static constexpr int OFF_ENDS = OFF_SCAN + 128 + 128;
    static constexpr int smem(int B) { return OFF_ENDS + B * (8 + (int)sizeof(Seq)) + 1024; }
    static_assert(B_END + 8 <= 256, "barrier block");
    static_assert(OFF_ENDS + LLAMA_PLAN_MAX_BATCH * (8 + (int)sizeof(Seq)) + 1024 <= 227 * 1024, "shared memory");
};

// Of a page: positions with NaN values per group; outside the pool; exponents
// (biased) of its largest key and value; whether its keys' sizes, its values'
// are wide apart
struct Notes {
    uint32_t nan[2][4];
    int bad, ke, ve, k_wide, v_wide, pad[3];
};
static_assert(sizeof(Notes) == 64, "notes");
// Of a wide page's rows: what brings a key back, and the exponent of a row's largest value
struct Rows {
    float k[PAGE], v[PAGE];
};
static_assert(sizeof(Rows) == 1024, "rows");
constexpr int WIDE = 8;              // exponents between the largest rows (of values: 64 channels of a row) and the smallest

// Products of one 16-deep step, D (+)= A B.  Shared-memory descriptors as
// their low words (address, leading offset): the high word is that of
// sw128_desc, so a step costs one addition per operand.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) { return ((addr & 0x3FFFFu) >> 4) | (lead << 16); }
__device__ __forceinline__ void umma_ss(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}\n" ::"r"(tmem_d),
        "r"(a_lo), "r"(b_lo), "r"(DESC_HI), "r"(idesc), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(tmem_d),
        "r"(tmem_a), "r"(b_lo), "r"(DESC_HI), "r"(idesc), "r"(accum)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// 16 columns of one TMEM lane per thread (warp-collective)
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ bool not_finite(uint32_t zs) {   // z or s
    return (zs & 0x7f80u) == 0x7f80u || (zs & 0x7f800000u) == 0x7f800000u;
}
// Exponent of a positive number, within what 2^(10 - exponent) and its inverse can be formed for
__device__ __forceinline__ int exponent(uint32_t bits) { return min(max((int)(bits >> 23), 30), 250); }
__device__ __forceinline__ float to_2_10(int e) { return __uint_as_float((uint32_t)(264 - e) << 23); }     // 2^(10 - exponent)
__device__ __forceinline__ float from_2_10(int e) { return __uint_as_float((uint32_t)(e - 10) << 23); }
constexpr uint32_t idesc_f16(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }

// A packed row's words to its place in a tile (row r), (z + n s) * f in fp16
template <int GR>
__device__ __forceinline__ void unpack_row(uint32_t tile, int r, const uint32_t (&w)[8 * GR], const uint32_t (&zs)[GR], float f) {
    constexpr uint32_t ONE = 0x3c003c00u, SIXTEENTH = 0x2c002c00u, M1024 = 0xe400e400u, M64 = 0xd400d400u;
#pragma unroll
    for (int gr = 0; gr < GR; ++gr) {
        const float zf = lo_bf16(zs[gr]) * f, sf = hi_bf16(zs[gr]) * f;
        const uint32_t s = pack_f16x2(sf, sf), z = pack_f16x2(zf, zf);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const uint32_t u = w[p * GR + gr], h = u >> 8;
            const uint32_t y0 = fma_f16x2(fma_f16x2((u & 0x000f000fu) | 0x64006400u, ONE, M1024), s, z);
            const uint32_t y1 = fma_f16x2(fma_f16x2((u & 0x00f000f0u) | 0x64006400u, SIXTEENTH, M64), s, z);
            const uint32_t y2 = fma_f16x2(fma_f16x2((h & 0x000f000fu) | 0x64006400u, ONE, M1024), s, z);
            const uint32_t y3 = fma_f16x2(fma_f16x2((h & 0x00f000f0u) | 0x64006400u, SIXTEENTH, M64), s, z);
            st_shared16(tile + gr * (128 * 128) + r * 128 + ((p ^ (r & 7)) << 4), y0, y1, y2, y3);
        }
    }
}

// The same as bf16 values, not scaled; no further from zero than the largest finite one (a call: rare, and out of the way)
template <int GR>
__device__ __noinline__ void unpack_row_bf16(uint32_t tile, int r, const uint32_t* w, const uint32_t* zs) {
    constexpr float MOST = 3.38953138925153547590e38f;
#pragma unroll 1
    for (int gr = 0; gr < GR; ++gr) {
        const float z = lo_bf16(zs[gr]), s = hi_bf16(zs[gr]);
#pragma unroll 1
        for (int p = 0; p < 8; ++p) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {        // codes i and i + 4: under the exponent of 2^23, less 2^23
                float v[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float n = __uint_as_float(((w[p * GR + gr] >> (4 * i + 16 * h)) & 15u) | 0x4b000000u) - 8388608.f;
                    v[h] = fminf(fmaxf(fmaf(n, s, z), -MOST), MOST);
                }
                y[i] = pack_bf16x2(v[0], v[1]);
            }
            st_shared16(tile + gr * (128 * 128) + r * 128 + ((p ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
        }
    }
}

// Rare pages stay out of the way of the others: calls, so that their registers and code do not count there.
// A column's scores, each times what brings its key back
__device__ __noinline__ void scores_wide(uint32_t s_addr, const float* k, float q_scale) {
#pragma unroll 1
    for (int c = 0; c < BKV / 32; ++c) {
        float s[32];
        tmem_ld32(s_addr + c * 32, s);
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] *= k[32 * c + i] * q_scale;
        tmem_st32(s_addr + c * 32, s);
    }
    tmem_st_wait();
}
// A column's weights 2^(score mul + shift), times f in two bf16 terms over the scores that they come from: 32 at a time,
// 16 columns of first terms and 16 of second ones.  Returns their sum (without f)
__device__ __noinline__ float weights_wide(uint32_t s_addr, int lim, float mul, float shift, float f) {
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < BKV / 32; ++c) {
        float w[32];
        tmem_ld32(s_addr + c * 32, w);
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            w[i] = ex2(fmaf(i + 32 * c <= lim ? w[i] : -INFINITY, mul, shift));
            part[i & 3] += w[i];
            w[i] *= f;
        }
        sum += (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = pack_bf16x2(w[2 * i], w[2 * i + 1]);
                w[2 * i] -= lo_bf16(p[i]);
                w[2 * i + 1] -= hi_bf16(p[i]);
            }
            tmem_st16(s_addr + c * 32 + t * 16, p);
        }
    }
    return sum;
}

// Pages that the columns up to `col` (of n G) see, one at least
__device__ __forceinline__ int pages_seen(const AttnArgs& a, const Seq& s, int col) {
    const int pos = s.len - s.n + min(col / a.G, s.n - 1);
    return pos < 0 ? 1 : pos / PAGE + 1;
}
__device__ __forceinline__ int items_of(const AttnArgs& a, const Seq& s) { return (s.n * a.G + ITEM - 1) / ITEM; }   // per head

// A CTA's stretch of one item: pages j0 .. j0 + nk - 1, of which tile x sees the first n[x]
struct Stretch {
    Seq sq;
    int b, head, item, pages;   // sequence, key/value head, item of the sequence, the item's pages
    int j0, nk, n0, n1;
    bool two;                   // the item has a second tile
    __device__ __forceinline__ int n(int x) const { return x ? n1 : n0; }
    __device__ __forceinline__ bool whole() const { return j0 == 0 && nk == pages; }
};
// The stretches of a range of units, one after another
struct Walk {
    const AttnArgs& a;
    const Seq* seqs;
    const long long* ends_;
    long long left;
    int b, head, item, j;
    __device__ __forceinline__ Walk(const AttnArgs& args, const Seq* sq, const long long* ends, long long u0, long long n)
        : a(args), seqs(sq), ends_(ends), left(n) {
        b = seq_of_unit(ends, a.B, u0);
        const long long before = b ? ends[b - 1] : 0, per_head = (ends[b] - before) / a.n_kv;
        head = (int)((u0 - before) / per_head);
        long long rest = (u0 - before) - head * per_head;
        for (item = 0;; ++item) {
            const int p = pages_seen(a, seqs[b], ITEM * (item + 1) - 1);
            if (rest < p) break;
            rest -= p;
        }
        j = (int)rest;
    }
    __device__ __forceinline__ Stretch get() const {
        Stretch s;
        s.sq = seqs[b];
        s.b = b;
        s.head = head;
        s.item = item;
        s.pages = pages_seen(a, s.sq, ITEM * (item + 1) - 1);
        s.two = ITEM * item + BQ < s.sq.n * a.G;
        s.j0 = j;
        s.nk = (int)min((long long)(s.pages - j), left);
        s.n0 = min(max(pages_seen(a, s.sq, ITEM * item + BQ - 1) - j, 0), s.nk);
        s.n1 = s.two ? s.nk : 0;
        return s;
    }
    __device__ __forceinline__ void next(const Stretch& s) {
        left -= s.nk;
        j += s.nk;
        if (j < s.pages || left <= 0) return;
        j = 0;
        if (++item < items_of(a, s.sq)) return;
        item = 0;
        if (++head < a.n_kv) return;
        head = 0;
        do ++b;
        while (ends_[b] == ends_[b - 1]);         // there are units left, so there is a sequence with some
    }
};

// What is joined at a CTA: the item that begins in it and goes on in the `more` CTAs after it (0: none)
struct TcJoin {
    int more, row0, head, col0, n_cols, pad[3];
};
// A part: outputs [hd / 4][columns][4], so that neighbouring columns (lanes) write and read neighbouring places, then
// (maximum, sum) [columns]
constexpr int part_floats(int hd) { return (hd + 2) * ITEM; }
__host__ __device__ constexpr int part_at(int col, int ch) { return (ch / 4 * ITEM + col) * 4 + ch % 4; }
__host__ __device__ constexpr int part_ml(int hd, int col) { return hd * ITEM + 2 * col; }
__host__ __device__ inline float* tc_parts(const AttnArgs& a) { return reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.work) + a.tc_offset); }
__device__ __forceinline__ TcJoin* tc_joins(const AttnArgs& a, int ctas, int hd) {
    return reinterpret_cast<TcJoin*>(tc_parts(a) + (size_t)ctas * 2 * part_floats(hd));
}

template <int HD>
__global__ void __launch_bounds__(NTHREADS, 1) kv4_attn_tc_kernel(const __grid_constant__ AttnArgs a) {
    using C = TCfg<HD>;
    constexpr int GR = HD / 64;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base, sK = base + C::OFF_K, sV = base + C::OFF_V, bars = base + C::OFF_BAR;
    const uint32_t q_full = bars + B_QFULL, q_empty = bars + B_QEMPTY, k_full = bars + B_KFULL, k_empty = bars + B_KEMPTY;
    const uint32_t v_full = bars + B_VFULL, v_empty = bars + B_VEMPTY;
    const uint32_t s_full = bars + B_SFULL;      // [2] S_x(n) in TMEM
    const uint32_t p_full = bars + B_PFULL;      // [2] P_x(n) in TMEM (and O_x rescaled); 128 arrivals
    const uint32_t pv_done = bars + B_PVDONE;    // [2] P_x(n) V done: S_x / P_x free, O_x current
    const uint32_t o_last = bars + B_OLAST;      // [2] the item's last P_x V done
    const uint32_t o_free = bars + B_OFREE;      // [2] O_x read out of TMEM; 128 arrivals
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_BAR + B_END);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Notes* notes = reinterpret_cast<Notes*>(gbase + C::OFF_NOTES);
    Rows* rows = reinterpret_cast<Rows*>(gbase + C::OFF_ROWS);
    long long* scan = reinterpret_cast<long long*>(gbase + C::OFF_SCAN);
    long long* ends = reinterpret_cast<long long*>(gbase + C::OFF_ENDS);
    Seq* seqs = reinterpret_cast<Seq*>(ends + a.B);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        mbar_init(q_full, 256);
        mbar_init(q_empty, 2);
        for (int i = 0; i < NS; ++i) {
            mbar_init(k_full + 8 * i, 128);
            mbar_init(k_empty + 8 * i, 2);
            mbar_init(v_full + 8 * i, 128);
            mbar_init(v_empty + 8 * i, 2);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full + 8 * x, 1);
            mbar_init(p_full + 8 * x, 128);
            mbar_init(pv_done + 8 * x, 1);
            mbar_init(o_last + 8 * x, 1);
            mbar_init(o_free + 8 * x, 128);
            mbar_init(bars + B_DRAIN + 8 * x, 1);
        }
        mbar_init(bars + B_TOPS, 4);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    const int beyond = columns_beyond<NTHREADS / 32>(a, seqs, ends, scan);
    const long long U = prefix<NTHREADS / 32>(a.B, ends, scan, [&](int i) {
        const Seq q = seqs[i];
        long long u = 0;
        if (many_columns(a, q, beyond))
            for (int k = 0; k < items_of(a, q); ++k) u += pages_seen(a, q, ITEM * (k + 1) - 1);
        return u * a.n_kv;
    });
    // two units per CTA at least, before another is used
    const int ctas = (int)min((long long)gridDim.x, (U + 1) / 2);
    TcJoin* join = tc_joins(a, gridDim.x, HD) + blockIdx.x;
    if (threadIdx.x == 0) join->more = 0;         // until the range's last stretch says otherwise
    if ((int)blockIdx.x >= ctas) return;
    const long long lo = U * blockIdx.x / ctas, hi = U * (blockIdx.x + 1) / ctas;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < SOFT0) {
        // ------------------------------------------------------ MMA issuer of tile x
        // the whole warp walks, one lane issues: operands that the compiler knows to be the same in all lanes are
        // formed in uniform registers, where the products take them from
        constexpr uint32_t IDESC_QK = idesc_f16(BKV);                  // K-major A and B
        constexpr uint32_t IDESC_PV = idesc_f16(HD) | (1u << 16);      // B (V) MN-major
        constexpr uint32_t IDESC_PV_WIDE = idesc_bf16(HD) | (1u << 16);
        const int x = __shfl_sync(0xffffffffu, warp, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t d_s = tm + 128u * x, d_o = tm + 256u + 128u * x;    // P over S
        const uint32_t q_lo = desc_lo(sQ + x * C::TILE, 1);
        const bool one = elect_one();
        bool ok = true;
        auto wait = [&](uint32_t bar, int n) {           // the barrier's n-th phase
            return (bool)__all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(n & 1), abort_flag, a.err));
        };
        int kv = 0, c = 0, nix = 0, ni = 0;              // pages so far, those that the tile sees, its stretches, the CTA's
        for (Walk walk(a, seqs, ends, lo, hi - lo); ok && walk.left > 0; ++ni) {
            const Stretch im = walk.get();
            walk.next(im);
            const int n = __shfl_sync(0xffffffffu, im.n(x), 0), nk = __shfl_sync(0xffffffffu, im.nk, 0);
            ok = wait(q_full, ni);
            for (int j = 0; ok && j < nk; ++j, ++kv) {
                const int st = kv % NS, use = kv / NS;
                const bool seen = j < n;
                // a page that the tile does not see is waited for all the same, so that its release is counted to it
                ok = wait(k_full + 8 * st, use) && (!seen || c == 0 || wait(pv_done + 8 * x, c - 1));
                if (!ok) break;
                if (one) {
                    if (seen) {
                        tc_fence_after();
                        const uint32_t k_lo = desc_lo(sK + st * C::TILE, 1);
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * C::REG + (kk & 3) * 32) >> 4;
                            umma_ss(d_s, q_lo + off, k_lo + off, IDESC_QK, kk > 0 ? 1u : 0u);
                        }
                        umma_commit(s_full + 8 * x);
                    }
                    umma_commit(k_empty + 8 * st);
                    if (j == nk - 1) umma_commit(q_empty);
                }
                __syncwarp();
                const bool wide = __shfl_sync(0xffffffffu, notes[kv % NF].v_wide, 0);       // there since k_full
                ok = wait(v_full + 8 * st, use) && (!seen || wait(p_full + 8 * x, c)) && (j > 0 || !seen || nix == 0 || wait(o_free + 8 * x, nix - 1));
                if (!ok) break;
                if (one) {
                    if (seen) {
                        tc_fence_after();
                        const uint32_t v_lo = desc_lo(sV + st * C::TILE, C::REG >> 4);                 // lead: the next 64 channels
                        if (wide) {                                                                    // 32 weights' first terms, their second
#pragma unroll
                            for (int kk = 0; kk < 2 * (BKV / 16); ++kk)
                                umma_ts(d_o, d_s + 32u * (kk >> 2) + 8u * ((kk >> 1) & 1) + 16u * (kk & 1), v_lo + (kk >> 1) * (2048u >> 4),
                                        IDESC_PV_WIDE, (j > 0 || kk > 0) ? 1u : 0u);
                        } else {
#pragma unroll
                            for (int kk = 0; kk < BKV / 16; ++kk) umma_ts(d_o, d_s + 8u * kk, v_lo + kk * (2048u >> 4), IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
                        }
                        umma_commit(pv_done + 8 * x);
                        if (j == n - 1) umma_commit(o_last + 8 * x);
                    }
                    umma_commit(v_empty + 8 * st);
                }
                __syncwarp();
                c += seen;
            }
            nix += n > 0;
        }
        if (one) mma_drain(bars + B_DRAIN + 8 * x);
    } else if (warp < UNPACK0) {
        // ------------------------------------------------------ queries, softmax, output
        const int x = (warp - SOFT0) >> 2, quarter = warp & 3;     // the quarter of TMEM's lanes that the warp can reach
        const int t_row = quarter * 32 + lane;           // column within the tile = TMEM lane
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const uint32_t o_addr = tmem + lane_addr + 256u + 128u * x, s_addr = tmem + lane_addr + 128u * x;
        bool ok = true;
        int sc = 0, nix = 0, ni = 0, kv0 = 0;
        for (Walk walk(a, seqs, ends, lo, hi - lo); ok && walk.left > 0; ++ni) {
            const Stretch im = walk.get();
            walk.next(im);
            const int gc = im.item * ITEM + x * BQ + t_row;
            const bool there = gc < im.sq.n * a.G;
            const int64_t row = im.sq.row0 + (there ? gc / a.G : 0);
            const int qh = im.head * a.G + (there ? gc % a.G : 0);
            if (ni > 0) ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (uint32_t)((ni - 1) & 1), abort_flag, a.err));
            if (!ok) break;
            float q_scale;                               // from products to base-2 scores, but for the page's factor
            {
                const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.q) + row * a.q_stride + (int64_t)qh * HD);
                uint4 w[HD / 8];
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    w[c] = there ? qp[c] : make_uint4(0, 0, 0, 0);
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu),
                                                 __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu)));
                }
                const uint32_t bits = max(top << 16, top & 0xffff0000u);
                const int e = exponent(bits);
                const float f = to_2_10(e);
                q_scale = bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : a.scale * from_2_10(e);
#pragma unroll
                for (int c = 0; c < HD / 8; ++c)
                    st_shared16(sQ + x * C::TILE + (c >> 3) * C::REG + t_row * 128 + (((c & 7) ^ (t_row & 7)) << 4),
                                pack_f16x2(lo_bf16(w[c].x) * f, lo_bf16(w[c].z) * f), pack_f16x2(hi_bf16(w[c].x) * f, hi_bf16(w[c].z) * f),
                                pack_f16x2(lo_bf16(w[c].y) * f, lo_bf16(w[c].w) * f), pack_f16x2(hi_bf16(w[c].y) * f, hi_bf16(w[c].w) * f));
                fence_async();
                mbar_arrive(q_full);
            }
            const int pos = im.sq.len - im.sq.n + (there ? gc / a.G : 0);      // sees positions 0 .. pos
            float m = -INFINITY, l = 0.f, poison[2] = {0.f, 0.f};
            int ve = 0, vtop = 0;                        // exponent that the outputs so far are scaled for, and the largest seen
            for (int j = 0; j < im.n(x); ++j, ++sc) {
                if (!__all_sync(0xffffffffu, mbar_wait(s_full + 8 * x, (uint32_t)(sc & 1), abort_flag, a.err))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const Notes& note = notes[(kv0 + j) % NF];
                const int lim = note.bad ? -1 : min(pos, im.sq.len - 1) - (im.j0 + j) * PAGE;   // last position of the page that is seen
                float mul = q_scale * from_2_10(note.ke);
                int page_ve = note.ve;
                const bool v_wide = note.v_wide;
                const Rows& own = rows[(kv0 + j) % NF];
                if (v_wide) {                            // of the values that the column sees
                    page_ve = 0;
                    for (int i = 0; i <= lim && i < BKV; ++i) page_ve = max(page_ve, (int)own.v[i]);
                    __syncwarp();                        // as many as a lane sees: together again for tensor memory
                }
                if (note.k_wide) {                       // scores brought back here
                    mul = 1.f;
                    scores_wide(s_addr, own.k, q_scale);
                }
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const uint4 v = *reinterpret_cast<const uint4*>(note.nan[gr]);
                    if (v.x | v.y | v.z | v.w) {
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int seen = lim + 1 - 32 * k;
                            const uint32_t mask = seen <= 0 ? 0u : seen >= 32 ? ~0u : (1u << seen) - 1u;
                            if (w[k] & mask) poison[gr] = __uint_as_float(0x7fc00000u);
                        }
                    }
                }
                // hidden scores are -inf and stay so: nothing of the page is seen, whatever the query; or the query's factor
                // and the keys' are so small that their product is 0 (scores of 0, up to 2^-97)
                if (lim < 0 || mul == 0.f) mul = __uint_as_float(1u << 23);
                // scores in halves: the second half's maximum, then the first half stays for its weights
                const bool cut = __any_sync(0xffffffffu, lim < BKV - 1);
                float sv[64], mx8[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) mx8[u] = -INFINITY;
                auto load = [&](int half, bool top) {
                    uint32_t* r = reinterpret_cast<uint32_t*>(sv);
                    TMEM_LD_X32(s_addr + 64 * half, r);
                    TMEM_LD_X32(s_addr + 64 * half + 32, (r + 32));
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    if (cut) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) sv[i] = i + 64 * half <= lim ? sv[i] : -INFINITY;
                    }
                    if (top) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) mx8[i & 7] = fmaxf(mx8[i & 7], sv[i]);
                    }
                };
                load(1, true);
                load(0, true);
                const float mt = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                       fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))) * mul;
                float corr = 1.f;
                bool rescale = false;
                if (m == -INFINITY) {
                    m = mt;                              // nothing but zeros accumulated yet
                } else if (mt > m + RESCALE_LOG2) {
                    corr = ex2(m - mt);
                    m = mt;
                    rescale = true;
                }
                // the values' factor: 2^(10 - page_ve) in them, so the weights carry 2^(page_ve - ve), 2^-8 .. 1: a page of
                // values of another size scales the outputs so far (fp32), up by 2^60 at most, instead of its weights (fp16)
                float resize = 1.f;
                if (page_ve > ve || (page_ve < ve - WIDE && page_ve > 0)) {
                    vtop = max(vtop, page_ve);
                    const int unit = max(page_ve, vtop - 60);
                    resize = ve == 0 ? 1.f : exp2f((float)(ve - unit));
                    ve = unit;
                    rescale |= resize != 1.f;
                }
                const float shift = m == -INFINITY ? 0.f : -m;
                // past 2^-40 the page adds nothing, but to the sum of weights
                const float carry = v_wide ? 0.f : (float)max(page_ve - ve, -40) + LIFT_LOG2;
                const float minus = shift + carry;
                float rs4[4] = {0.f, 0.f, 0.f, 0.f};
                if (v_wide) {                            // values in bf16, weights in two terms of it: they bring any value to the outputs' scale
                    rs4[0] = weights_wide(s_addr, lim, mul, shift, ve == 0 ? 0.f : to_2_10(ve) * LIFT);     // 0: nothing seen so far
                } else
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (half == 1) load(1, false);
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float p0 = ex2(fmaf(sv[2 * i], mul, minus)), p1 = ex2(fmaf(sv[2 * i + 1], mul, minus));
                        pk[i] = pack_f16x2(p0, p1);
                        rs4[i & 3] += p0 + p1;
                    }
                    asm volatile(
                        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
                        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(s_addr + 32 * half),
                        "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7]), "r"(pk[8]),
                        "r"(pk[9]), "r"(pk[10]), "r"(pk[11]), "r"(pk[12]), "r"(pk[13]), "r"(pk[14]), "r"(pk[15]), "r"(pk[16]),
                        "r"(pk[17]), "r"(pk[18]), "r"(pk[19]), "r"(pk[20]), "r"(pk[21]), "r"(pk[22]), "r"(pk[23]), "r"(pk[24]),
                        "r"(pk[25]), "r"(pk[26]), "r"(pk[27]), "r"(pk[28]), "r"(pk[29]), "r"(pk[30]), "r"(pk[31])
                        : "memory");
                }
                const float rs = (rs4[0] + rs4[1]) + (rs4[2] + rs4[3]);
                tmem_st_wait();
                // a warp with a moved maximum rescales its rows of O_x: the previous P_x V has completed
                // (S_x(j) was issued after it)
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                    for (int c = 0; c < HD / 32; ++c) {
                        float ov[32];
                        tmem_ld32(o_addr + c * 32, ov);
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] *= corr * resize;
                        tmem_st32(o_addr + c * 32, ov);
                    }
                    tmem_st_wait();
                }
                l = fmaf(rs, exp2f(-carry), l * corr);
                tc_fence_before();
                mbar_arrive(p_full + 8 * x);
            }
            if (!ok) break;
            const bool any = im.n(x) > 0, whole = im.whole();
            if (any) {
                ok = __all_sync(0xffffffffu, mbar_wait(o_last + 8 * x, (uint32_t)(nix & 1), abort_flag, a.err));
                if (!ok) break;
                tc_fence_after();
            }
            // to the output if this CTA has all of the item, else as a part: its beginning in slot 1, else in slot 0
            const float back = (whole ? inverse(l) : 1.f) * (ve == 0 ? 1.f : from_2_10(ve) * (1.f / LIFT));
            bf16* dst = static_cast<bf16*>(a.o) + row * ((int64_t)a.H * HD) + (int64_t)qh * HD;
            float* part = tc_parts(a) + ((size_t)blockIdx.x * 2 + (im.j0 == 0)) * part_floats(HD);
            const int col = x * BQ + t_row;
            if (any || there) {
#pragma unroll 1
                for (int c = 0; c < HD / 32; ++c) {
                    float ov[32];
                    if (any) {
                        tmem_ld32(o_addr + c * 32, ov);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = 0.f;
                    }
                    const float bad = poison[(c * 32) / 64];
                    if (there) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            float y[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[(i >> 1) + 4 * (i & 1)] = fmaf(ov[8 * u + i], back, bad);   // c0 c4 c1 c5 ..
                            if (whole) {
                                *reinterpret_cast<uint4*>(dst + c * 32 + 8 * u) = make_uint4(
                                    pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
                            } else {
                                *reinterpret_cast<float4*>(part + part_at(col, c * 32 + 8 * u)) = make_float4(y[0], y[1], y[2], y[3]);
                                *reinterpret_cast<float4*>(part + part_at(col, c * 32 + 8 * u + 4)) = make_float4(y[4], y[5], y[6], y[7]);
                            }
                        }
                    }
                }
                if (!whole && there) {
                    *reinterpret_cast<float2*>(part + part_ml(HD, col)) = make_float2(m, l);
                }
            }
            if (any) {
                tc_fence_before();
                mbar_arrive(o_free + 8 * x);
                ++nix;
            }
            // for the second kernel: an item that begins here and goes on
            if (x == 0 && t_row == 0 && im.j0 == 0 && !whole) {
                const long long end = hi - im.nk + im.pages;          // this stretch is the range's last
                TcJoin t{};
                t.more = (int)((end * ctas + U - 1) / U) - 1 - (int)blockIdx.x;
                t.row0 = im.sq.row0;
                t.head = im.head;
                t.col0 = im.item * ITEM;
                t.n_cols = min(im.sq.n * a.G - t.col0, ITEM);
                *join = t;
            }
            kv0 += im.nk;
        }
    } else {
        // ------------------------------------------------------ unpacking: a position per thread
        const int r = threadIdx.x - UNPACK0 * 32;
        bool ok = true;
        int kt = 0;
        // [page parity][largest key, value, smallest key, value][warp], behind the scan
        uint32_t* tops = reinterpret_cast<uint32_t*>(scan) + 32;
        for (Walk walk(a, seqs, ends, lo, hi - lo); ok && walk.left > 0;) {
            const Stretch im = walk.get();
            walk.next(im);
            const int nk = im.nk;
            uint32_t kw[8 * GR], vw[8 * GR], kz[GR], vz[GR];
            int bad = 0;
            auto page_of = [&](int i) {
                const int j = im.j0 + i;
                return i < nk && j * PAGE < im.sq.len ? a.table[(int64_t)im.b * a.pps + j] : -1;
            };
            auto fetch = [&](int i, int page) {          // this position's rows of the i-th page, zeros where it holds nothing
                const int j = im.j0 + i;
                const bool want = i < nk && j * PAGE + r < im.sq.len;
                const bool have = page >= 0 && page < a.n_pages;
                bad = i < nk && j * PAGE < im.sq.len && !have;
#pragma unroll
                for (int k = 0; k < 8 * GR; ++k) kw[k] = vw[k] = 0;
#pragma unroll
                for (int k = 0; k < GR; ++k) kz[k] = vz[k] = 0;
                if (want && have) {
                    const uint8_t* p = a.pool + blk_offset(page, a.n_kv, im.head, r, HD);
                    const uint8_t* v = p + half_bytes(HD);
                    const int q = r % BLK;
#pragma unroll
                    for (int i = 0; i < 2 * GR; ++i) {
                        const uint4 u = *(reinterpret_cast<const uint4*>(p + q * code_bytes(HD)) + i);
                        const uint4 w = *(reinterpret_cast<const uint4*>(v + q * code_bytes(HD)) + i);
                        kw[4 * i] = u.x; kw[4 * i + 1] = u.y; kw[4 * i + 2] = u.z; kw[4 * i + 3] = u.w;
                        vw[4 * i] = w.x; vw[4 * i + 1] = w.y; vw[4 * i + 2] = w.z; vw[4 * i + 3] = w.w;
                    }
#pragma unroll
                    for (int i = 0; i < GR; ++i) {
                        kz[i] = *(reinterpret_cast<const uint32_t*>(p + BLK * code_bytes(HD)) + q * GR + i);
                        vz[i] = *(reinterpret_cast<const uint32_t*>(v + BLK * code_bytes(HD)) + q * GR + i);
                    }
                }
            };
            int page = page_of(0);
            fetch(0, page);
            page = page_of(1);
            for (int j = 0; j < nk; ++j, ++kt) {
                const int st = kt % NS;
                const uint32_t par = ((kt / NS) & 1) ^ 1u;
                uint32_t w[8 * GR], z[GR], nv[8 * GR], nz[GR];
#pragma unroll
                for (int i = 0; i < 8 * GR; ++i) {
                    w[i] = kw[i];
                    nv[i] = vw[i];
                }
#pragma unroll
                for (int i = 0; i < GR; ++i) {
                    z[i] = kz[i];
                    nz[i] = vz[i];
                }
                const int now_bad = bad;
                if (bad && r == 0) atomicOr(a.err, LLAMA_DEVERR_INPUT);
                fetch(j + 1, page);                      // the next page's rows, and the page after it
                page = page_of(j + 2);
                ok = __all_sync(0xffffffffu, mbar_wait(k_empty + 8 * st, par, abort_flag, a.err));
                if (!ok) break;
                uint32_t kt_top = 0, vt_top = 0, vt_least = ~0u;     // bits of |z| + 15 s, which no value passes
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const unsigned nan = __ballot_sync(0xffffffffu, not_finite(nz[gr]));
                    if (not_finite(nz[gr])) nz[gr] = 0;
                    if (lane == 0) notes[kt % NF].nan[gr][r / 32] = nan;
                    if (!not_finite(z[gr])) kt_top = max(kt_top, __float_as_uint(fabsf(lo_bf16(z[gr])) + 15.f * hi_bf16(z[gr])));
                    else z[gr] = 0x7fc07fc0u;
                    const uint32_t v = __float_as_uint(fabsf(lo_bf16(nz[gr])) + 15.f * hi_bf16(nz[gr]));
                    vt_top = max(vt_top, v);
                    vt_least = min(vt_least, v - 1u);                // not of zeros
                }
                const uint32_t k_max = __reduce_max_sync(0xffffffffu, kt_top), v_max = __reduce_max_sync(0xffffffffu, vt_top);
                const uint32_t k_min = __reduce_min_sync(0xffffffffu, kt_top - 1u), v_min = __reduce_min_sync(0xffffffffu, vt_least);
                uint32_t* top = tops + (kt & 1) * 16;
                if (lane == 0) {
                    top[r / 32] = k_max;
                    top[4 + r / 32] = v_max;
                    top[8 + r / 32] = k_min;
                    top[12 + r / 32] = v_min;
                    mbar_arrive(bars + B_TOPS);
                }
                ok = __all_sync(0xffffffffu, mbar_wait(bars + B_TOPS, (uint32_t)(kt & 1), abort_flag, a.err));   // all four warps'
                if (!ok) break;
                int ke = exponent(max(max(top[0], top[1]), max(top[2], top[3])));
                const int vee = exponent(max(max(top[4], top[5]), max(top[6], top[7])));
                const bool k_wide = exponent(min(min(top[8], top[9]), min(top[10], top[11]))) < ke - WIDE;
                const bool v_wide = exponent(min(min(top[12], top[13]), min(top[14], top[15]))) < vee - WIDE;
                if (r == 0) {
                    notes[kt % NF].bad = now_bad;
                    notes[kt % NF].ke = ke;
                    notes[kt % NF].ve = vee;
                    notes[kt % NF].k_wide = k_wide;
                    notes[kt % NF].v_wide = v_wide;
                }
                if (k_wide) {
                    ke = exponent(kt_top);
                    rows[kt % NF].k[r] = from_2_10(ke);
                }
                if (v_wide) rows[kt % NF].v[r] = (float)exponent(vt_top);
                unpack_row<GR>(sK + st * C::TILE, r, w, z, to_2_10(ke));
                fence_async();
                mbar_arrive(k_full + 8 * st);
                ok = __all_sync(0xffffffffu, mbar_wait(v_empty + 8 * st, par, abort_flag, a.err));
                if (!ok) break;
                if (v_wide) {
                    uint32_t wv[8 * GR], wz[GR];
#pragma unroll
                    for (int i = 0; i < 8 * GR; ++i) wv[i] = nv[i];
#pragma unroll
                    for (int i = 0; i < GR; ++i) wz[i] = nz[i];
                    unpack_row_bf16<GR>(sV + st * C::TILE, r, wv, wz);
                } else {
                    unpack_row<GR>(sV + st * C::TILE, r, nv, nz, to_2_10(vee));
                }
                fence_async();
                mbar_arrive(v_full + 8 * st);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the parts of the items that span CTAs: block (c, y) takes 32 columns
// of the item that begins in the first kernel's CTA c and goes on.  A thread
// has four channels of a column at a time; eight lanes write 64 bytes of one.
constexpr int JOIN_THREADS = 256, JOIN_COLS = 32;

template <int HD>
__global__ void __launch_bounds__(JOIN_THREADS) kv4_join_tc_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int QUADS = HD / 4 / 8;                    // per thread: channels 4 (lane % 8) + 32 i ..
    __shared__ float top[JOIN_COLS], sum[JOIN_COLS];     // the columns' maximum and inverse sum
    pdl_launch_dependents();
    pdl_wait();
    const TcJoin j = tc_joins(a, gridDim.x, HD)[blockIdx.x];
    const int col0 = blockIdx.y * JOIN_COLS;
    if (j.more <= 0 || col0 >= j.n_cols) return;
    // part k: the item's beginning here, then the CTAs after
    auto part = [&](int k) { return tc_parts(a) + ((size_t)(blockIdx.x + k) * 2 + (k == 0)) * part_floats(HD); };
    const int local = threadIdx.x / 8, q = threadIdx.x % 8, col = min(col0 + local, j.n_cols - 1);
    {                                                    // eight lanes look through a column's parts
        float M = -INFINITY, L = 0.f;
        for (int k = q; k <= j.more; k += 8) M = fmaxf(M, part(k)[part_ml(HD, col)]);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (q == 0) {
            for (int k = 0; k <= j.more; ++k) {          // in order: the sum does not depend on the split into lanes
                const float2 ml = *reinterpret_cast<const float2*>(part(k) + part_ml(HD, col));
                L = fmaf(ml.y, ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - M), L);
            }
            top[local] = M;
            sum[local] = inverse(L);
        }
        __syncwarp();
    }
    const float M = top[local], inv = sum[local];
    float4 y[QUADS];
#pragma unroll
    for (int i = 0; i < QUADS; ++i) y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = 0; k <= j.more; ++k) {
        const float* p = part(k);
        const float2 ml = *reinterpret_cast<const float2*>(p + part_ml(HD, col));
        const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - M);
#pragma unroll
        for (int i = 0; i < QUADS; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(p + part_at(col, 4 * q + 32 * i));
            y[i].x = fmaf(v.x, f, y[i].x);
            y[i].y = fmaf(v.y, f, y[i].y);
            y[i].z = fmaf(v.z, f, y[i].z);
            y[i].w = fmaf(v.w, f, y[i].w);
        }
    }
    if (col0 + local >= j.n_cols) return;
    const int gc = j.col0 + col;
    bf16* o = static_cast<bf16*>(a.o) + (int64_t)(j.row0 + gc / a.G) * ((int64_t)a.H * HD) + (j.head * a.G + gc % a.G) * HD + 4 * q;
#pragma unroll
    for (int i = 0; i < QUADS; ++i)
        *reinterpret_cast<uint2*>(o + 32 * i) = make_uint2(pack_bf16x2(y[i].x * inv, y[i].y * inv), pack_bf16x2(y[i].z * inv, y[i].w * inv));
}

template <int HD>
int run(const AttnArgs& a, cudaStream_t st) {
    using C = TCfg<HD>;
    static PerDeviceOnce once;
    int rc = once_per_device(once, []() -> int {
        LLAMA_CUDA_TRY(cudaFuncSetAttribute(kv4_attn_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(LLAMA_PLAN_MAX_BATCH)));
        return (int)LLAMA_OK;
    });
    if (rc) return rc;
    const int ctas = std::min(tc_num_sms(), STEP_MAX_CTAS);
    launch_pdl(kv4_attn_tc_kernel<HD>, dim3(ctas), dim3(NTHREADS), C::smem(a.B), st, a);
    LLAMA_LAUNCH_CHECK();
    launch_pdl(kv4_join_tc_kernel<HD>, dim3(ctas, ITEM / JOIN_COLS), dim3(JOIN_THREADS), 0, st, a);
    LLAMA_LAUNCH_CHECK();
    return LLAMA_OK;
}

}  // namespace

uint64_t attention_kv4_tc_work_bytes(int hd) {
    return (uint64_t)STEP_MAX_CTAS * (2 * part_floats(hd) * sizeof(float) + sizeof(TcJoin));
}

int launch_attention_kv4_tc(const void* args, int hd, cudaStream_t st) {
    const AttnArgs& a = *static_cast<const AttnArgs*>(args);
    return hd == 128 ? run<128>(a, st) : run<64>(a, st);
}
