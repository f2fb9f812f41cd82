// Low-rank adapters of many requests at once, beside a shared projection:
//   y[r, :] += scale_a * (x[r, :] A_a^T) B_a^T      for every row r of adapter a
// with A_a [rank, d] and B_a [n, rank].  Rows come grouped by adapter, in
// tiles of up to 64 rows (llama_op_batch_plan, or any caller's grouping).
//
// Two kernels.  `down` forms h = x A^T: an item is a tile's rows x 64 ranks
// and a slice of d; the slice's partial goes to the workspace in fp32 (no
// atomics: slices are added in order later).  `up` adds the slices, scales,
// and multiplies with B_a; its results are added to y where y is held, in L2
// (four floats per reduction), so that no load of y is waited for.
//
// Bound: HBM (x once, y twice, A and B once per adapter); at rank 64 the
// products are 50 flops per byte, which mma.sync covers (the tensor pipe is
// busy a third of the time), and tiles of 64 ragged rows would leave tcgen05's
// 128-row tiles half empty.  What counts is bytes in flight: `down` streams
// 64-channel pieces through a four-stage cp.async ring, whose copies gather
// the rows.  8192 rows x 4096 -> 4096, 4 adapters of rank 64: 90 us (the bytes
// alone: 52 us), of them `up` 59 (y at 4.6 TB/s), `down` 30; 700 rows, 13824 ->
// 5120, 13 of rank 8: 22 us (8 us); 32 rows, 16 of rank 16: 8.3 us, latency.
//
// Precision: y is fp32, so h must not be rounded to bf16: it enters the
// second product as three bf16 terms (24 bits).  fp32 operands are split the
// same way, on both sides, and the six products that matter are summed: fp32
// accuracy from the same instructions.
#include "common.cuh"
#include "kernels.h"

namespace {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int SUB = 32;              // rows of a down item (fp32)
constexpr int RANKS = 64;            // ranks of a down item
constexpr int COLS = 256;            // columns of y per step of an up CTA: 32 per warp

struct LoraArgs {
    const void* x;
    const void* A;
    const void* B;
    const float* scale;
    float* y;
    const int32_t* rows;
    const int4* tiles;
    const int32_t* n_tiles;
    float* h;                        // [slices][M][rank], row = place in `rows`
    int M, d, n, rank, n_adapters, max_tiles;
    int slices, slice_len;           // slice_len: channels, a multiple of 64
    int steps;                       // column steps of an up CTA
    int64_t ldx, ldy;
    int* err;
};

// A tile that can be used: adapter and rows inside what they index
struct Tile {
    int adapter, start, count;
};
__device__ __forceinline__ Tile tile_of(const LoraArgs& a, int i) {
    Tile t{0, 0, 0};
    const int n = *a.n_tiles;
    if (n < 0 || n > a.max_tiles) atomicOr(a.err, LLAMA_DEVERR_INPUT);
    if (i >= min(n, a.max_tiles)) return t;
    const int4 v = a.tiles[i];
    if (v.x < 0 || v.x >= a.n_adapters || v.z < 0 || v.z > LLAMA_LORA_TILE || v.y < 0 || v.y > a.M - v.z) {
        atomicOr(a.err, LLAMA_DEVERR_INPUT);
        return t;
    }
    return Tile{v.x, v.y, v.z};
}
// Row of x and y at a place of the list, or -1
__device__ __forceinline__ int row_of(const LoraArgs& a, int place) {
    const int r = a.rows[place];
    if (r >= 0 && r < a.M) return r;
    atomicOr(a.err, LLAMA_DEVERR_INPUT);
    return -1;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x, y as n bf16 pairs, each the rounding of what the ones before left over
template <int N>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t* t, int stride) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i * stride] = pack_bf16x2(x, y);
        const float2 f = unpack_bf16x2(t[i * stride]);
        x -= f.x;
        y -= f.y;
    }
}
// 8 neighbouring fp32 channels as 4 pairs in three terms
struct Terms {
    uint32_t r[3][4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 12; ++i) r[i / 4][i % 4] = 0;
    }
    __device__ __forceinline__ void load(const float* p) {
        const float4 u = *(reinterpret_cast<const float4*>(p)), v = *(reinterpret_cast<const float4*>(p) + 1);
        split_pair<3>(u.x, u.y, &r[0][0], 4);
        split_pair<3>(u.z, u.w, &r[0][1], 4);
        split_pair<3>(v.x, v.y, &r[0][2], 4);
        split_pair<3>(v.z, v.w, &r[0][3], 4);
    }
};

// Products of two 16-deep steps (8 channels per lane) of split operands: the
// terms whose weights add up to less than 2^-24 of the product are left out.
// The matrix instructions cut their sums instead of rounding them to nearest:
// over a long chain that shows in the fifth digit.  So the steps are summed by
// themselves, smallest terms first, and added in fp32.
__device__ __forceinline__ void mma_steps(float (&d)[4], const uint32_t (&a0)[3][4], const uint32_t (&a1)[3][4],
                                          const uint32_t (&b)[3][4]) {
    float part[4] = {};
#pragma unroll
    for (int w = 2; w >= 0; --w)
#pragma unroll
        for (int i = 0; i <= w; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                mma_bf16(part, a0[i][2 * s], a1[i][2 * s], a0[i][2 * s + 1], a1[i][2 * s + 1], b[w - i][2 * s], b[w - i][2 * s + 1]);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] += part[e];
}

// bf16: h of a tile's rows x 64 ranks over one slice of d.  Ranks are the m of
// the product, rows its n; warp (i, j) of 4 x 2 has 16 ranks and 32 rows.
// Rows of 64 channels sit in shared memory as 8 chunks of 16 bytes, chunk c
// of row r at c ^ (r % 8), which ldmatrix reads without conflicts.
constexpr int PIECE = 64;            // channels per stage
constexpr int STAGES = 4;            // 64 KB
constexpr int HALF = LLAMA_LORA_TILE * PIECE * 2;     // bytes of a stage's x (and of its A)

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {   // zeros when off
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__global__ void __launch_bounds__(THREADS, 2) lora_down_bf16_kernel(const __grid_constant__ LoraArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];
    pdl_launch_dependents();
    pdl_wait();
    const int rank_blocks = (a.rank + RANKS - 1) / RANKS;
    int item = blockIdx.x;
    const int slice = item % a.slices;
    item /= a.slices;
    const int rb = item % rank_blocks;
    const Tile tile = tile_of(a, item / rank_blocks);
    if (tile.count <= 0) return;
    const int ranks = min(a.rank - rb * RANKS, RANKS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // copies: this thread's chunk of rows r, r + 32 of x and of A
    const int r = threadIdx.x >> 3, chunk = threadIdx.x & 7;
    const bf16* src[4];
    bool on[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int place = r + 32 * i;
        const int row = place < tile.count ? row_of(a, tile.start + place) : -1;
        on[i] = row >= 0;
        src[i] = static_cast<const bf16*>(a.x) + (on[i] ? row * a.ldx : 0) + chunk * 8;
        on[2 + i] = place < ranks;
        src[2 + i] = static_cast<const bf16*>(a.A) + ((int64_t)tile.adapter * a.rank + rb * RANKS + (on[2 + i] ? place : 0)) * a.d + chunk * 8;
    }
    const bool need[4] = {true, tile.count > 32, true, ranks > 32};     // rows 32 .. 63 that some warp reads
    const uint32_t base = smem_addr(ring);
    const uint32_t dst = base + r * 128 + ((chunk ^ (r & 7)) << 4);     // row r + 32 has the same r % 8
    const int k0 = slice * a.slice_len, k1 = min(a.d, k0 + a.slice_len);
    const int pieces = k1 > k0 ? (k1 - k0 + PIECE - 1) / PIECE : 0;
    auto fetch = [&](int p, uint32_t stage) {
        if (p < pieces) {
            const int k = k0 + p * PIECE;
            const bool in = k + chunk * 8 < k1;                          // d is a multiple of 8
            const uint32_t to = dst + stage;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (need[i]) copy16(to + (i >> 1) * HALF + (i & 1) * 32 * 128, in ? src[i] + k : src[i], in && on[i]);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // a piece is summed by itself and added in fp32: the tensor cores' additions do not round to nearest, which shows
    // in the seventh digit of y (32 rows, rank 16: 9e-8 of y; cut every 4 pieces 2.1e-7, in the same time)
    float total[4][4] = {};
    const int wi = warp & 3, wj = warp >> 2;
    const bool works = wi * 16 < ranks && wj * 32 < tile.count;
    const int ar = wi * 16 + (lane & 15), br = wj * 32 + (lane & 7) + ((lane >> 4) << 3);
    for (int p = 0; p < STAGES - 1; ++p) fetch(p, p * 2 * HALF);
    uint32_t stage = 0, next = (STAGES - 1) * 2 * HALF;                  // of piece p, and of the one fetched beside it
    for (int p = 0; p < pieces; ++p) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        __syncthreads();                          // piece p is there, and piece p - 1 has been read
        fetch(p + STAGES - 1, next);
        const uint32_t xs = base + stage, as = xs + HALF;
        next = stage;
        stage = stage == (STAGES - 1) * 2 * HALF ? 0 : stage + 2 * HALF;
        if (!works) continue;
        float acc[4][4] = {};
#pragma unroll
        for (int ks = 0; ks < PIECE / 16; ++ks) {
            uint32_t fa[4], fb[2][4];
            ldmatrix4(fa, as + ar * 128 + (((2 * ks + (lane >> 4)) ^ (ar & 7)) << 4));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                ldmatrix4(fb[h], xs + (br + 16 * h) * 128 + (((2 * ks + ((lane >> 3) & 1)) ^ (br & 7)) << 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_bf16(acc[j], fa[0], fa[1], fa[2], fa[3], fb[j >> 1][2 * (j & 1)], fb[j >> 1][2 * (j & 1) + 1]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) total[j / 4][j % 4] += acc[j / 4][j % 4];
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!works) return;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int place = wj * 32 + j * 8 + 2 * t + (e & 1), c = wi * 16 + g + 8 * (e >> 1);
            if (place < tile.count && c < ranks)
                a.h[((int64_t)slice * a.M + tile.start + place) * a.rank + rb * RANKS + c] = total[j][e];
        }
}

// fp32: h of up to 32 rows x 64 ranks over one slice of d, operands straight
// from global memory in split terms: the k order of a product is free, so a
// lane takes 8 neighbouring channels of a row as its part of two 16-deep
// steps.  8 warps take 32-channel pieces in turn and meet in shared memory.
__global__ void __launch_bounds__(THREADS) lora_down_f32_kernel(const __grid_constant__ LoraArgs a) {
    extern __shared__ float sum[];                // [WARPS][SUB rows][RANKS + 1]
    pdl_launch_dependents();
    pdl_wait();
    const int rank_blocks = (a.rank + RANKS - 1) / RANKS;
    const int subs = LLAMA_LORA_TILE / SUB;
    int item = blockIdx.x;
    const int slice = item % a.slices;
    item /= a.slices;
    const int rb = item % rank_blocks;
    item /= rank_blocks;
    const int sub = item % subs;
    const Tile tile = tile_of(a, item / subs);
    const int rows = min(tile.count - sub * SUB, SUB);
    if (rows <= 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nt = (rows + 7) / 8, mt = (min(a.rank - rb * RANKS, RANKS) + 15) / 16;
    const float* xr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int place = j * 8 + g;
        const int r = place < rows ? row_of(a, tile.start + sub * SUB + place) : -1;
        xr[j] = r >= 0 ? static_cast<const float*>(a.x) + r * a.ldx : nullptr;
    }
    const float* A = static_cast<const float*>(a.A) + ((int64_t)tile.adapter * a.rank + rb * RANKS) * a.d;
    float acc[4][4][4];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i / 16][i / 4 % 4][i % 4] = 0.f;
    const int k_end = min(a.d, (slice + 1) * a.slice_len);
    for (int k = slice * a.slice_len + warp * 32; k < k_end; k += WARPS * 32) {
        const int ch = k + 8 * t;
        const bool in = ch < k_end;               // d is a multiple of 8
        Terms xb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            xb[j].zero();
            if (j < nt && in && xr[j]) xb[j].load(xr[j] + ch);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= mt) break;
            Terms a0, a1;
            a0.zero();
            a1.zero();
            const int r0 = i * 16 + g;
            if (in && rb * RANKS + r0 < a.rank) a0.load(A + (int64_t)r0 * a.d + ch);
            if (in && rb * RANKS + r0 + 8 < a.rank) a1.load(A + (int64_t)(r0 + 8) * a.d + ch);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < nt) mma_steps(acc[i][j], a0.r, a1.r, xb[j].r);
        }
    }
    float* mine = sum + warp * SUB * (RANKS + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i < mt && j < nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mine[(j * 8 + 2 * t + (e & 1)) * (RANKS + 1) + i * 16 + g + 8 * (e >> 1)] = acc[i][j][e];
    __syncthreads();
    const int ranks = min(a.rank - rb * RANKS, RANKS);
    for (int e = threadIdx.x; e < rows * ranks; e += THREADS) {
        const int r = e / ranks, c = e - r * ranks;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += sum[(w * SUB + r) * (RANKS + 1) + c];
        a.h[((int64_t)slice * a.M + tile.start + sub * SUB + r) * a.rank + rb * RANKS + c] = v;
    }
}

// Four neighbouring floats of y, added where they are held (L2): every element
// is added to once per call, so the order of additions is no question
__device__ __forceinline__ void add4(float* p, float x, float y, float z, float w) {
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

// h of a tile into shared memory: its slices added, times the scale, in three
// bf16 terms [term][row][rank rounded up to 32], rows padded by 16 bytes
constexpr int TERMS = 3;
template <int DEEP, int SLICES>
__device__ __forceinline__ void gather_quads(const LoraArgs& a, const Tile& tile, uint8_t* hs, int K, int pitch) {
    const float scale = a.scale[tile.adapter];
    const int rows = (tile.count + 15) / 16 * 16, quads = K / 4;
    for (int e0 = threadIdx.x; e0 < rows * quads; e0 += THREADS * DEEP) {
        float4 v[DEEP];
        const float* p[DEEP];
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            const int e = e0 + d * THREADS, r = e / quads, c = (e - r * quads) * 4;
            v[d] = make_float4(0.f, 0.f, 0.f, 0.f);
            p[d] = r < tile.count && c < a.rank ? a.h + ((int64_t)tile.start + r) * a.rank + c : nullptr;
        }
#pragma unroll SLICES
        for (int s = 0; s < a.slices; ++s) {
#pragma unroll
            for (int d = 0; d < DEEP; ++d)
                if (p[d]) {
                    const float4 u = *reinterpret_cast<const float4*>(p[d] + (int64_t)s * a.M * a.rank);
                    v[d].x += u.x;
                    v[d].y += u.y;
                    v[d].z += u.z;
                    v[d].w += u.w;
                }
        }
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            const int e = e0 + d * THREADS, r = e / quads, c = (e - r * quads) * 4;
            if (e >= rows * quads) break;
            uint32_t lo[TERMS], hi[TERMS];
            split_pair<TERMS>(v[d].x * scale, v[d].y * scale, lo, 1);
            split_pair<TERMS>(v[d].z * scale, v[d].w * scale, hi, 1);
#pragma unroll
            for (int i = 0; i < TERMS; ++i) *reinterpret_cast<uint2*>(hs + (i * LLAMA_LORA_TILE + r) * pitch + c * 2) = make_uint2(lo[i], hi[i]);
        }
    }
}

// Four ranks at a time, 16 of those in flight: over the slices when they are
// many (4096 x 4096, 700 rows, 13 adapters of rank 8, 16 slices: 16.5 us
// against 18.1 for the whole operator), over places too when they are not
// (8192 rows, rank 64, 3 slices: 91.7 us against 93.9)
__device__ __forceinline__ void gather_h(const LoraArgs& a, const Tile& tile, uint8_t* hs, int K, int pitch) {
    if (a.slices > 4) gather_quads<1, 16>(a, tile, hs, K, pitch);
    else gather_quads<4, 4>(a, tile, hs, K, pitch);
}

// bf16: y of a tile's rows, BLOCK columns per step.  Rows are the m of the
// product, columns its n.  A step's part of B comes through a two-stage
// cp.async ring, the next one while this one is used (one stage for ranks
// past 128); with up to 16 rows all
// warps share the columns, with more they share the rows too.  Column e of
// the n-tile j stands for column 4 (e / 2) + 2 j + e % 2 of 16, so that a
// lane's results of two n-tiles are four neighbouring columns of y.
constexpr int BLOCK = 128;
constexpr int up_pitch(int rank) { return (rank + 31) / 32 * 64 + 16; }      // bytes of a row of h and of B in shared memory
constexpr int up_stages(int rank) { return rank > 128 ? 1 : 2; }             // two no longer fit
constexpr int up_smem(int rank) { return (TERMS * LLAMA_LORA_TILE + up_stages(rank) * BLOCK) * up_pitch(rank); }

template <int NB>
__global__ void __launch_bounds__(THREADS) lora_up_bf16_kernel(const __grid_constant__ LoraArgs a) {
    extern __shared__ __align__(128) uint8_t hs[];
    pdl_launch_dependents();
    pdl_wait();
    const Tile tile = tile_of(a, blockIdx.y);
    if (tile.count <= 0) return;
    const int K = (a.rank + 31) / 32 * 32, pitch = up_pitch(a.rank);
    const uint32_t h_base = smem_addr(hs), b_base = h_base + TERMS * LLAMA_LORA_TILE * pitch;
    const bf16* B = static_cast<const bf16*>(a.B) + (int64_t)tile.adapter * a.n * a.rank;
    const int first = blockIdx.x * a.steps, steps = min(a.steps, (a.n + BLOCK - 1) / BLOCK - first);
    const int chunks = K / 8;                     // 16-byte pieces of a row of B (zeros past the rank)
    auto fetch = [&](int step) {
        if (step < steps)
            for (int e = threadIdx.x; e < BLOCK * chunks; e += THREADS) {
                const int col = e / chunks, c = e - col * chunks, n = (first + step) * BLOCK + col;
                const bool on = n < a.n && c * 8 < a.rank;
                copy16(b_base + (step % NB * BLOCK + col) * pitch + c * 16, on ? B + (int64_t)n * a.rank + c * 8 : B, on);
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int mts = (tile.count + 15) / 16;
    const int groups = mts == 1 ? 1 : mts == 2 ? 2 : 4;         // of rows; 8 / groups warps share the columns
    const int mt = warp % groups, col0 = warp / groups * 16 * groups;
    int r[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int place = mt * 16 + g + 8 * hh;
        r[hh] = place < tile.count ? row_of(a, tile.start + place) : -1;
    }
    gather_h(a, tile, hs, K, pitch);
    // ldmatrix rows of B: the column that n-tile row (lane % 8) of tile (lane / 16) stands for, k half (lane / 8) % 2
    const int e = lane & 7, bcol = 4 * (e / 2) + 2 * (lane >> 4) + e % 2;
    for (int step = 0; step < steps; ++step) {
        if (NB > 1 || step > 0) fetch(NB > 1 ? step + 1 : step);
        asm volatile("cp.async.wait_group %0;" ::"n"(NB - 1) : "memory");
        __syncthreads();                          // this step's columns (and, before the first, h)
        if (mt < mts) {
            float acc[4][2][4];                   // [16 columns][n-tile][.]
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i / 8][i / 4 % 2][i % 4] = 0.f;
            const uint32_t b_row = b_base + (step % NB * BLOCK + col0 + bcol) * pitch + ((lane >> 3) & 1) * 16;
            const uint32_t h_row = h_base + (mt * 16 + (lane & 15)) * pitch + (lane >> 4) * 16;
            for (int k = 0; k < K; k += 16) {
                uint32_t h[TERMS][4];
#pragma unroll
                for (int i = 0; i < TERMS; ++i) ldmatrix4(h[i], h_row + i * LLAMA_LORA_TILE * pitch + k * 2);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= groups) break;
                    uint32_t b[4];
                    ldmatrix4(b, b_row + q * 16 * pitch + k * 2);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // smallest terms first; many steps (one stage of B) are summed by themselves and added in fp32
                        // (rank 256: error 6.7e-7 -> 1.2e-7, 1024 x 4096: 116 -> 121 us; rank 128 without: 3.5e-7)
                        float part[4] = {};
                        float(&d)[4] = NB == 1 ? part : acc[q][j];
#pragma unroll
                        for (int i = TERMS - 1; i >= 0; --i) mma_bf16(d, h[i][0], h[i][1], h[i][2], h[i][3], b[2 * j], b[2 * j + 1]);
                        if constexpr (NB == 1)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[q][j][e] += part[e];
                    }
                }
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                if (r[hh] < 0) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = (first + step) * BLOCK + col0 + q * 16 + 4 * t;
                    if (q < groups && n < a.n)    // n is a multiple of 4
                        add4(a.y + r[hh] * a.ldy + n, acc[q][0][2 * hh], acc[q][0][2 * hh + 1], acc[q][1][2 * hh], acc[q][1][2 * hh + 1]);
                }
            }
        }
        __syncthreads();                          // before the stage is filled again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// fp32: the same with B split into three terms as it is loaded
__global__ void __launch_bounds__(THREADS) lora_up_f32_kernel(const __grid_constant__ LoraArgs a) {
    extern __shared__ __align__(128) uint8_t hs[];
    __shared__ int row[LLAMA_LORA_TILE];
    pdl_launch_dependents();
    pdl_wait();
    const Tile tile = tile_of(a, blockIdx.y);
    if (tile.count <= 0) return;
    const int K = (a.rank + 31) / 32 * 32, pitch = up_pitch(a.rank);
    const int mts = (tile.count + 15) / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (threadIdx.x < LLAMA_LORA_TILE) row[threadIdx.x] = threadIdx.x < tile.count ? row_of(a, tile.start + threadIdx.x) : -1;
    gather_h(a, tile, hs, K, pitch);
    __syncthreads();
    const float* B = static_cast<const float*>(a.B) + (int64_t)tile.adapter * a.n * a.rank;
    for (int step = 0; step < a.steps; ++step) {
        const int n0 = (blockIdx.x * a.steps + step) * COLS + warp * 32;
        if (n0 >= a.n) break;
        float acc[4][2][2][4];                    // [16 rows][16 columns][n-tile][.]
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i / 16][i / 8 % 2][i / 4 % 2][i % 4] = 0.f;
        for (int k = 0; k < K; k += 32) {
            Terms b[2][2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = n0 + q * 16 + 4 * (g / 2) + 2 * j + g % 2;
                    b[q][j].zero();
                    if (col < a.n && k + 8 * t < a.rank) b[q][j].load(B + (int64_t)col * a.rank + k + 8 * t);
                }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                if (mt >= mts) break;
                uint32_t h0[TERMS][4], h1[TERMS][4];
#pragma unroll
                for (int i = 0; i < TERMS; ++i) {
                    const uint8_t* p = hs + (i * LLAMA_LORA_TILE + mt * 16 + g) * pitch + (k + 8 * t) * 2;
                    const uint4 u = *reinterpret_cast<const uint4*>(p), v = *reinterpret_cast<const uint4*>(p + 8 * pitch);
                    h0[i][0] = u.x; h0[i][1] = u.y; h0[i][2] = u.z; h0[i][3] = u.w;
                    h1[i][0] = v.x; h1[i][1] = v.y; h1[i][2] = v.z; h1[i][3] = v.w;
                }
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int j = 0; j < 2; ++j) mma_steps(acc[mt][q][j], h0, h1, b[q][j].r);
            }
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int r = mt < mts ? row[mt * 16 + g + 8 * hh] : -1;
                if (r < 0) continue;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int col = n0 + q * 16 + 4 * t;
                    if (col < a.n)                // n is a multiple of 4
                        add4(a.y + r * a.ldy + col, acc[mt][q][0][2 * hh], acc[mt][q][0][2 * hh + 1], acc[mt][q][1][2 * hh],
                             acc[mt][q][1][2 * hh + 1]);
                }
            }
    }
}

constexpr int MAX_SLICES = 16;

template <typename Kernel>
int allow_smem(Kernel k, int bytes) {
    LLAMA_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    return LLAMA_OK;
}

int run(bool is_bf16, LoraArgs& a, cudaStream_t st) {
    constexpr int DOWN_BF16 = STAGES * 2 * HALF, DOWN_F32 = WARPS * SUB * (RANKS + 1) * (int)sizeof(float);
    static PerDeviceOnce once;
    int rc = once_per_device(once, []() -> int {
        int e;
        if ((e = allow_smem(lora_down_bf16_kernel, DOWN_BF16)) || (e = allow_smem(lora_down_f32_kernel, DOWN_F32)) ||
            (e = allow_smem(lora_up_bf16_kernel<1>, up_smem(LLAMA_LORA_MAX_RANK))) ||
            (e = allow_smem(lora_up_bf16_kernel<2>, up_smem(128))) || (e = allow_smem(lora_up_f32_kernel, up_smem(LLAMA_LORA_MAX_RANK))))
            return e;
        return (int)LLAMA_OK;
    });
    if (rc) return rc;
    const int rank_blocks = (a.rank + RANKS - 1) / RANKS;
    const unsigned items = (unsigned)a.max_tiles * rank_blocks * a.slices;
    if (is_bf16) launch_pdl(lora_down_bf16_kernel, dim3(items), dim3(THREADS), (size_t)DOWN_BF16, st, a);
    else launch_pdl(lora_down_f32_kernel, dim3(items * (LLAMA_LORA_TILE / SUB)), dim3(THREADS), (size_t)DOWN_F32, st, a);
    LLAMA_LAUNCH_CHECK();
    // every CTA of a tile adds the slices again, so a tile gets as many CTAs as fill the SMs four times, and in bf16 each
    // at least two steps, the second's B on its way beside the first (24 tiles, n 5120: 24.7 us for the whole operator,
    // twice: 26.2, once: 33.5; one step of 32 rows on 16 adapters, n 4096: 10.4 us against 9.3).  fp32: twice, one CTA
    // per SM at a time (24 tiles of rank 8, 2048 x 5120: 28.8 us, once: 37.8; 18 tiles of rank 64, 5120 x 5120: 127 us,
    // once: 116, four times: 122; 9 tiles, 1024 x 1024: 23.0, two steps each: 31.7)
    const int cols = ceil_div(a.n, is_bf16 ? BLOCK : COLS), fill = (is_bf16 ? 4 : 2) * 148;
    const int want = a.max_tiles < fill ? fill / a.max_tiles : 1;
    a.steps = ceil_div(cols, want < cols ? want : cols);
    if (is_bf16 && a.steps < 2) a.steps = 2;
    const dim3 grid(ceil_div(cols, a.steps), a.max_tiles);
    const size_t smem = (size_t)up_smem(a.rank);
    if (!is_bf16) launch_pdl(lora_up_f32_kernel, grid, dim3(THREADS), smem, st, a);
    else if (up_stages(a.rank) == 2) launch_pdl(lora_up_bf16_kernel<2>, grid, dim3(THREADS), smem, st, a);
    else launch_pdl(lora_up_bf16_kernel<1>, grid, dim3(THREADS), smem, st, a);
    LLAMA_LAUNCH_CHECK();
    return LLAMA_OK;
}

// Slices of d: four items per SM (two run at a time), four pieces of 64
// channels each at least.  700 rows x 13824, rank 8, 13 adapters, and 8192 rows
// x 4096, rank 64 (the whole operator): 21.9 and 89.4 us; three items per SM:
// 22.8 and 95.3; two, with 6 stages: 31.3 and 92.3; three CTAs in 80 registers
// each: 24.3 and 91.8, four in 64: 26.9 and 93.9.
int slices_of(int max_tiles, int rank, int d) {
    const int items = max_tiles * ((rank + RANKS - 1) / RANKS);
    int s = (4 * 148) / items;
    s = s < 1 ? 1 : s;
    const int most = (d + 4 * PIECE - 1) / (4 * PIECE);
    s = s > MAX_SLICES ? MAX_SLICES : s;
    return s > most ? most : s;
}

}  // namespace

uint64_t lora_work_bytes(int M, int rank) { return (uint64_t)MAX_SLICES * M * rank * sizeof(float); }

int launch_lora(int dtype, const void* x, int64_t ldx, const void* A, const void* B, const float* scale, float* y, int64_t ldy,
                const int32_t* rows, const int32_t* tiles, const int32_t* n_tiles, int max_tiles, int M, int d, int n, int rank,
                int n_adapters, float* work, int* err, cudaStream_t st) {
    LoraArgs a;
    a.x = x;
    a.A = A;
    a.B = B;
    a.scale = scale;
    a.y = y;
    a.rows = rows;
    a.tiles = reinterpret_cast<const int4*>(tiles);
    a.n_tiles = n_tiles;
    a.h = work;
    a.M = M;
    a.d = d;
    a.n = n;
    a.rank = rank;
    a.n_adapters = n_adapters;
    a.max_tiles = max_tiles;
    a.slices = slices_of(max_tiles, rank, d);
    a.slice_len = ceil_div(ceil_div(d, a.slices), PIECE) * PIECE;
    a.steps = 1;
    a.ldx = ldx;
    a.ldy = ldy;
    a.err = err;
    return run(dtype == LLAMA_BF16, a, st);
}
