// Keys and values into the 4-bit paged cache, and back out of it.
//
// Append: per (row, head, 64 channels)
//   z = the largest bf16 value not above min x
//   s = the smallest bf16 value not below (max x - z) / 15
//   n = the nearest whole number to (x - z) / s (ties to even), 0 where s = 0
// so every value is at most s / 2 from z + n s.  A group that holds a NaN or
// an infinity gets z = s = NaN: it reads back as NaN and nothing else does.
//
// The result is that of 64-bit arithmetic, exactly: the quotients are formed
// in fp32 and only those within 2^-12 of a border are looked at again, with
// exact arithmetic, because fp64 divisions for every value would cost more
// than the memory traffic.
//
// A thread takes 16 channels (two words of codes) of one row's keys and of its
// values, four neighbouring lanes share a group and reduce by two shuffles;
// lanes walk a row's heads in order, so loads are contiguous, and a row's
// codes leave as whole 32-byte sectors.  The row's data is requested beside
// its slot, not after it.
//
// 8192 rows x 32 heads of 128, bf16 (134 MB in, 38 MB of cache): 73 us for
// the two in a row: append at 3.4 TB/s, bound by the instructions of the
// quantiser (320 for 16 values; issue slots 77% busy), read at 6.2 TB/s, bound
// by HBM.  Keys and values in threads of their own, each finding its row, slot
// and place: 89 us for the two.  Every value converted, divided and clamped on
// its own: 189 us; so the group's arithmetic is shared by 16 values, codes are
// packed by fused multiply-adds, and only rare groups take the long way.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace {

constexpr int THREADS = 128;         // append and read as above: 73 us, with 64 and 256 threads 81 and 76
constexpr int PER = 16;              // channels per thread

// n / d for n < 2^31 by a product and a shift (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994)
struct FastDiv {
    uint32_t d, m, l;
    explicit FastDiv(uint32_t div) : d(div), l(0) {
        while ((1ull << l) < div) ++l;
        m = (uint32_t)(((1ull << 32) * ((1ull << l) - div)) / div + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> l; }
};

// 32 bytes at once where rows start on 32 bytes (W), else 16 twice
template <bool W>
__device__ __forceinline__ void load32(const void* p, uint32_t (&u)[8]) {
    if constexpr (W) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                     : "l"(p)
                     : "memory");
    } else {
        const uint4 a = *(static_cast<const uint4*>(p)), b = *(static_cast<const uint4*>(p) + 1);
        u[0] = a.x; u[1] = a.y; u[2] = a.z; u[3] = a.w;
        u[4] = b.x; u[5] = b.y; u[6] = b.z; u[7] = b.w;
    }
}
template <bool W>
__device__ __forceinline__ void store32(void* p, const uint32_t (&u)[8]) {
    if constexpr (W) {
        asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                     "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "l"(p)
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        static_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A thread's 16 channels of a row, and the lowest and highest of the 64 of its
// group (NaN if one of them is)
template <typename T> struct Chunk;
template <> struct Chunk<bf16> {
    uint32_t u[8];
    template <bool W>
    __device__ __forceinline__ void load(const bf16* p) { load32<W>(p, u); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const {
        return __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
    }
    __device__ __forceinline__ void range(float& lo, float& hi) const {
        uint32_t a = u[0], b = u[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            a = min2_nan(a, u[i]);
            b = max2_nan(b, u[i]);
        }
        b ^= 0x80008000u;                        // (lowest, minus the highest): both by the same minimum
        uint32_t r = min2_nan(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
        r = min2_nan(r, __shfl_xor_sync(0xffffffffu, r, 1));
        r = min2_nan(r, __shfl_xor_sync(0xffffffffu, r, 2));
        lo = __uint_as_float(r << 16);
        hi = -__uint_as_float(r & 0xffff0000u);
    }
};
template <> struct Chunk<float> {
    uint32_t u[16];
    template <bool W>
    __device__ __forceinline__ void load(const float* p) {
        uint32_t a[8];
        load32<W>(p, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = a[i];
        load32<W>(p + 8, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[8 + i] = a[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(u[i]); }
    __device__ __forceinline__ void range(float& lo, float& hi) const {
        float a = at(0), b = -at(0);
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            a = min_nan(a, at(i));
            b = min_nan(b, -at(i));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            a = min_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
            b = min_nan(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
        lo = a;
        hi = -b;
    }
};

// The largest bf16 not above x (finite; no lower than the lowest finite bf16)
__device__ __forceinline__ float bf16_floor(float x) {
    uint32_t b = __float_as_uint(x);
    if ((b & 0xffffu) == 0) return x;
    b = (b & 0x80000000u) ? (b | 0xffffu) + 1u : b;      // away from zero below it, towards zero above it
    return fmaxf(__uint_as_float(b & 0xffff0000u), __uint_as_float(0xff7f0000u));
}

// The smallest bf16 not below r (in 64 bits), 0 for a negative r
__device__ __noinline__ float bf16_ceil64(double r) {
    if (!(r > 0.0)) return 0.f;
    uint32_t b = __float_as_uint(__double2float_rz(r)) & 0xffff0000u;    // not above r
    if ((double)__uint_as_float(b) < r) b += 0x10000u;
    return __uint_as_float(b);
}

__device__ __noinline__ uint32_t code64(float x, float z, float s) {
    const double n = rint(((double)x - (double)z) / (double)s);
    return (uint32_t)(n < 0.0 ? 0.0 : n > 15.0 ? 15.0 : n);
}

// The code of one value whose quotient t (within 2^-12) lies next to the
// border between two codes.  bf16 values meet borders often (one in some
// hundred quotients of short numbers is a half exactly), so they are decided
// in fp32 where x - z is exact: the sign of (x - z) - border * s, which one
// fused multiply-add gives exactly.
__device__ __forceinline__ uint32_t code_at_border(float x, float z, float s, float t) {
    const float d = x - z, e = d - x;
    if (!(((x - (d - e)) - (z + e)) == 0.f && fabsf(t) < 16.f)) return code64(x, z, s);   // x - z is rounded
    const float below = floorf(t), over = fmaf(-(below + 0.5f), s, d);
    // t may lie on the other side of a whole number than the quotient, not of the border
    const float n = over > 0.f ? below + 1.f : over < 0.f ? below : 2.f * rintf(0.5f * (below + 0.5f));
    return (uint32_t)n;
}

// A thread's two words of codes, and z | s << 16 of its group; src: where the
// thread's channels came from
template <typename T>
__device__ __forceinline__ uint32_t quantise(const Chunk<T>& c, const T* src, uint32_t (&w)[2]) {
    float lo, hi;
    c.range(lo, hi);
    w[0] = w[1] = 0;
    if (!(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY)) return 0x7fc07fc0u;
    // a zero offset is +0, whichever zero the minimum is
    const float z = (sizeof(T) == 2 ? lo : bf16_floor(lo)) + 0.f;
    const float r = (hi - z) * (1.f / 15.f);     // within 2^-22 of the quotient, relative
    const uint32_t rb = __float_as_uint(r);
    float s;
    if ((rb & 0xffffu) - 16u < 0x10000u - 32u && r > 1e-30f && r < 1e38f) s = __uint_as_float((rb & 0xffff0000u) + 0x10000u);
    else s = bf16_ceil64(((double)hi - (double)z) / 15.0);
    const uint32_t zs = (__float_as_uint(z) >> 16) | (__float_as_uint(s) & 0xffff0000u);
    if (s == 0.f) return zs;
    // (x - z) / s as x / s - z / s: with |z / s| < 2^9 both products and the sum are within 2^-13 of it
    const float inv = 1.f / s, off = -z * inv;
    constexpr float ROUND = 12582912.f;          // 1.5 * 2^23: adding it rounds to whole numbers
    unsigned next = 0;                           // values next to a border
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = fmaf(c.at(8 * h + i), inv, off);
            n[i] = (t + ROUND) - ROUND;
            if (!(fabsf(t - n[i]) < 0.5f - 2.44140625e-4f)) next |= 1u << (8 * h + i);
        }
        // four codes as one number below 2^16, exact in fp32, then its bits
        const float a = fmaf(n[3], 4096.f, fmaf(n[2], 256.f, fmaf(n[1], 16.f, n[0]))) + 8388608.f;
        const float b = fmaf(n[7], 4096.f, fmaf(n[6], 256.f, fmaf(n[5], 16.f, n[4]))) + 8388608.f;
        w[h] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
    }
    if (!(fabsf(off) < 512.f && lo >= z)) {      // out of the short way's range: every value by itself
        next = 0;
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            uint32_t& word = i < 8 ? w[0] : w[1];
            word = (word & ~(15u << (4 * (i & 7)))) | (code64(to_f32(src[i]), z, s) << (4 * (i & 7)));
        }
    }
    while (next) {
        const int i = __ffs(next) - 1;
        next &= next - 1;
        const float x = to_f32(src[i]);
        uint32_t& word = i < 8 ? w[0] : w[1];
        word = (word & ~(15u << (4 * (i & 7)))) | (code_at_border(x, z, s, fmaf(x, inv, off)) << (4 * (i & 7)));
    }
    return zs;
}

struct StoreArgs {
    const int32_t* slots;
    uint8_t* pool;
    int64_t k_stride, v_stride;   // elements between rows
    int64_t n_slots;              // 128 * pages
    unsigned items;               // rows * n_kv * hd / 16
    FastDiv per;                  // n_kv * hd / 16: pieces of a row's keys
    int n_kv;
    int* err;
};

// A thread's piece: 16 channels of a row's keys, and of its values
struct Piece {
    unsigned row;
    int ch;
};
__device__ __forceinline__ Piece piece_of(const StoreArgs& a, unsigned item) {
    const unsigned row = a.per.div(item);
    return Piece{row, (int)(item - row * a.per.d) * PER};
}
// The keys' words and scale pair in the cache (the values' are half_bytes on);
// false for a row that is not stored
template <int HD>
__device__ __forceinline__ bool locate(const StoreArgs& a, const Piece& p, int32_t slot, int64_t& word, int64_t& pair) {
    constexpr int G = kv4::groups(HD);
    if (slot < 0 || slot >= a.n_slots) {
        if (slot >= a.n_slots) atomicOr(a.err, LLAMA_DEVERR_INPUT);
        return false;
    }
    const int head = p.ch / HD, c = p.ch % HD;
    const int64_t base = kv4::blk_offset(slot / kv4::PAGE, a.n_kv, head, slot % kv4::PAGE, HD);
    const int r = slot % kv4::BLK, g = c / kv4::GROUP;
    word = base + r * kv4::code_bytes(HD) + (c % kv4::GROUP / 8 * G + g) * 4;     // the second word is G words on
    pair = base + kv4::BLK * kv4::code_bytes(HD) + (r * G + g) * 4;
    return true;
}

template <typename T, int HD, bool W>
__global__ void __launch_bounds__(THREADS) kv4_append_kernel(const T* k, const T* v, const __grid_constant__ StoreArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const unsigned item = blockIdx.x * THREADS + threadIdx.x;
    const bool on = item < a.items;              // the four lanes of a group are on together
    Chunk<T> c[2];
    c[0].zero();
    c[1].zero();
    Piece p{0, 0};
    int32_t slot = -1;
    const T* src[2] = {k, v};
    if (on) {
        p = piece_of(a, item);
        slot = a.slots[p.row];
        src[0] += p.row * a.k_stride + p.ch;
        src[1] += p.row * a.v_stride + p.ch;
        c[0].template load<W>(src[0]);
        c[1].template load<W>(src[1]);
    }
    int64_t word = 0, pair = 0;
    const bool stored = on && locate<HD>(a, p, slot, word, pair);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        uint32_t w[2];
        const uint32_t zs = quantise(c[which], src[which], w);
        if (stored) {
            uint8_t* half = a.pool + which * kv4::half_bytes(HD);
            *reinterpret_cast<uint32_t*>(half + word) = w[0];
            *reinterpret_cast<uint32_t*>(half + word + 4 * kv4::groups(HD)) = w[1];
            if ((threadIdx.x & 3) == 0) *reinterpret_cast<uint32_t*>(half + pair) = zs;
        }
    }
}

// 16 values of a thread's two words
template <typename T, bool W>
__device__ __forceinline__ void put16(T* dst, const uint32_t (&w)[2], uint32_t zs) {
    const float z = __uint_as_float(zs << 16), s = __uint_as_float(zs & 0xffff0000u);
    const float most = __uint_as_float(sizeof(T) == 4 ? 0x7f7fffffu : 0x7f7f0000u);   // the largest finite T
    // the step is rounded up: at the very end of the range z + 15 s may pass what T holds
    const bool end = fabsf(z) + 15.f * s > most;
    uint32_t u[8];
    if constexpr (sizeof(T) == 2) {
        // codes i and i + 4 of a word as bf16 128 + n (n under 128's exponent), n by an exact subtraction, z + n s
        // by one fused multiply-add, rounded once
        const uint32_t ss = __byte_perm(zs, 0, 0x3232), zz = __byte_perm(zs, 0, 0x1010);
        constexpr uint32_t E = 0x43004300u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t n;
                asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(((w[h] >> (4 * i)) & 0x000f000fu) | E), "r"(E));
                asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y[i]) : "r"(n), "r"(ss), "r"(zz));
            }
            u[4 * h] = __byte_perm(y[0], y[1], 0x5410);
            u[4 * h + 1] = __byte_perm(y[2], y[3], 0x5410);
            u[4 * h + 2] = __byte_perm(y[0], y[1], 0x7632);
            u[4 * h + 3] = __byte_perm(y[2], y[3], 0x7632);
        }
        if (end) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {        // an infinity becomes the largest finite value
                if ((u[i] & 0x7fffu) == 0x7f80u) u[i] -= 1u;
                if ((u[i] & 0x7fff0000u) == 0x7f800000u) u[i] -= 0x10000u;
            }
        }
        store32<W>(dst, u);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {        // the code under the exponent of 2^23, less 2^23
                float y = fmaf(__uint_as_float(((w[h] >> (4 * i)) & 15u) | 0x4b000000u) - 8388608.f, s, z);
                if (end && fabsf(y) > most) y = copysignf(most, y);
                u[i] = __float_as_uint(y);
            }
            store32<W>(dst + 8 * h, u);
        }
    }
}

template <typename T, int HD, bool W>
__global__ void __launch_bounds__(THREADS) kv4_read_kernel(T* k, T* v, const __grid_constant__ StoreArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const unsigned item = blockIdx.x * THREADS + threadIdx.x;
    if (item >= a.items) return;
    const Piece p = piece_of(a, item);
    uint32_t w[2][2] = {}, zs[2] = {};           // a row that is not in the cache reads as zeros
    int64_t word, pair;
    if (locate<HD>(a, p, a.slots[p.row], word, pair)) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint8_t* half = a.pool + which * kv4::half_bytes(HD);
            w[which][0] = *reinterpret_cast<const uint32_t*>(half + word);
            w[which][1] = *reinterpret_cast<const uint32_t*>(half + word + 4 * kv4::groups(HD));
            zs[which] = *reinterpret_cast<const uint32_t*>(half + pair);
        }
    }
    put16<T, W>(k + p.row * a.k_stride + p.ch, w[0], zs[0]);
    put16<T, W>(v + p.row * a.v_stride + p.ch, w[1], zs[1]);
}

// Rows start on 32 bytes
bool wide(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int esz) {
    return ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | (uintptr_t)(k_stride * esz) | (uintptr_t)(v_stride * esz)) & 31u) == 0;
}

template <typename T, int HD>
int append(const void* k, const void* v, const StoreArgs& a, cudaStream_t st) {
    const dim3 grid(ceil_div(a.items, THREADS));
    if (wide(k, v, a.k_stride, a.v_stride, sizeof(T)))
        launch_pdl(kv4_append_kernel<T, HD, true>, grid, dim3(THREADS), 0, st, (const T*)k, (const T*)v, a);
    else
        launch_pdl(kv4_append_kernel<T, HD, false>, grid, dim3(THREADS), 0, st, (const T*)k, (const T*)v, a);
    LLAMA_LAUNCH_CHECK();
    return LLAMA_OK;
}
template <typename T, int HD>
int read(void* k, void* v, const StoreArgs& a, cudaStream_t st) {
    const dim3 grid(ceil_div(a.items, THREADS));
    if (wide(k, v, a.k_stride, a.v_stride, sizeof(T)))
        launch_pdl(kv4_read_kernel<T, HD, true>, grid, dim3(THREADS), 0, st, (T*)k, (T*)v, a);
    else
        launch_pdl(kv4_read_kernel<T, HD, false>, grid, dim3(THREADS), 0, st, (T*)k, (T*)v, a);
    LLAMA_LAUNCH_CHECK();
    return LLAMA_OK;
}

}  // namespace

int launch_kv4_append(int dtype, const void* k, const void* v, const int32_t* slots, uint8_t* pool, int rows, int n_kv,
                      int hd, int64_t k_stride, int64_t v_stride, int64_t n_slots, int* err, cudaStream_t st) {
    const unsigned per = (unsigned)(n_kv * hd / PER);
    const StoreArgs a{slots, pool, k_stride, v_stride, n_slots, (unsigned)rows * per, FastDiv(per), n_kv, err};
    if (dtype == LLAMA_BF16) return hd == 128 ? append<bf16, 128>(k, v, a, st) : append<bf16, 64>(k, v, a, st);
    return hd == 128 ? append<float, 128>(k, v, a, st) : append<float, 64>(k, v, a, st);
}

int launch_kv4_read(int dtype, void* k, void* v, const int32_t* slots, const uint8_t* pool, int rows, int n_kv, int hd,
                    int64_t k_stride, int64_t v_stride, int64_t n_slots, int* err, cudaStream_t st) {
    const unsigned per = (unsigned)(n_kv * hd / PER);
    const StoreArgs a{slots, const_cast<uint8_t*>(pool), k_stride, v_stride, n_slots, (unsigned)rows * per, FastDiv(per), n_kv, err};
    if (dtype == LLAMA_BF16) return hd == 128 ? read<bf16, 128>(k, v, a, st) : read<bf16, 64>(k, v, a, st);
    return hd == 128 ? read<float, 128>(k, v, a, st) : read<float, 64>(k, v, a, st);
}
