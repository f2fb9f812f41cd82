// The plan of one serving step, built on the device from request lengths:
// which requests run, their rows, the pages they get, the cache slot and the
// position of every row, and the rows grouped by adapter.
//
// Everything follows from prefix sums over the requests (tokens, pages,
// adapter rows), so one CTA of 1024 threads, a request per thread, does the
// sums; the per-row and per-page tables are then filled row-parallel by a
// binary search in those sums.  The work is a few kilobytes: latency bounds
// it.  Up to FUSED_ROWS rows the same CTA fills them too (one launch); past
// that a second kernel spreads the rows over the SMs.  64 requests, 8
// adapters, 512, 2048, 4096 and 16384 rows: 5.0, 5.8, 6.9 and 11.1 us in the
// one CTA, 6.4, 6.2, 6.4 and 6.2 us with the second kernel.
//
// Sums saturate at 2^31 - 1: saturating addition of non-negative numbers is
// associative, and every capacity they are compared with is smaller.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace {

constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int FUSED_ROWS = 2048;
constexpr unsigned CAP = 0x7fffffffu;

__device__ __forceinline__ unsigned sat(unsigned a, unsigned b) { return min(a + b, CAP); }

// Inclusive saturating prefix sums of two values over the CTA
__device__ __forceinline__ void scan2(unsigned& a, unsigned& b, uint2* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a = sat(a, x);
            b = sat(b, y);
        }
    }
    if (lane == 31) part[warp] = make_uint2(a, b);
    __syncthreads();
    uint2 t = part[lane];                        // 32 warps: one total per lane
    unsigned x = t.x, y = t.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x = sat(x, u);
            y = sat(y, v);
        }
    }
    const unsigned bx = __shfl_sync(0xffffffffu, x, max(warp - 1, 0)), by = __shfl_sync(0xffffffffu, y, max(warp - 1, 0));
    if (warp > 0) {
        a = sat(a, bx);
        b = sat(b, by);
    }
    __syncthreads();                             // part is free again
}

// First index in ends[0..n) whose value is above x (n if none)
template <typename T>
__device__ __forceinline__ int above(const T* ends, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int)ends[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Row r of the step: its request, position and slot, and its place among its
// adapter's rows.  Per request: first[b], its first position less its first
// row, and lora[b], the place of its first row (-1 without adapter).
__device__ __forceinline__ void fill_row(const llama_batch_plan& p, const int* cu, const int* first, const int* lora,
                                         int r, int rows, int lora_rows, int* err) {
    int seq = -1, pos = -1, slot = -1;
    if (r < rows) {
        seq = above(cu + 1, p.B, r);
        pos = first[seq] + r;
        const int page = *(volatile const int*)(p.d_table + (int64_t)seq * p.pages_per_seq + pos / kv4::PAGE);
        if (page >= 0 && page < p.n_pages) slot = page * kv4::PAGE + pos % kv4::PAGE;
        else atomicOr(err, LLAMA_DEVERR_INPUT);
        if (p.n_adapters > 0 && lora[seq] >= 0) p.d_lora_rows[lora[seq] + r - cu[seq]] = r;
    }
    p.d_slots[r] = slot;
    p.d_pos[r] = pos;
    p.d_seq[r] = seq;
    if (p.n_adapters > 0 && r >= lora_rows) p.d_lora_rows[r] = -1;
}

// d_work of the plan: [0] rows, [1] rows with an adapter, then first[B] and
// lora[B] of fill_row (kept here and not read again from d_past, which may be
// the buffer that d_kv_len writes: the lengths of the next step)
__global__ void __launch_bounds__(THREADS) batch_plan_kernel(const __grid_constant__ llama_batch_plan p, int fused, int* err) {
    extern __shared__ int dyn[];                 // [warps in use][n_adapters] rows per (warp, adapter)
    __shared__ uint2 part[WARPS];
    __shared__ int cu[THREADS + 1], page_end[THREADS], held_of[THREADS], lora[THREADS], first[THREADS];
    __shared__ int a_start[LLAMA_PLAN_MAX_ADAPTERS], a_rows[LLAMA_PLAN_MAX_ADAPTERS], a_tiles[LLAMA_PLAN_MAX_ADAPTERS];
    __shared__ int n_new_s[THREADS];
    __shared__ int total_rows, total_pages, total_lora, total_tiles;
    pdl_launch_dependents();
    const int t = threadIdx.x, B = p.B, A = p.n_adapters, warps = (B + 31) / 32;
    if (t == 0) total_rows = total_pages = total_lora = total_tiles = 0;
    for (int i = t; i < warps * A; i += THREADS) dyn[i] = 0;
    pdl_wait();
    int past = 0, fresh = 0, adapter = -1;
    bool right = false;
    if (t < B) {
        past = p.d_past[t];
        fresh = p.d_new[t];
        if (A > 0) adapter = p.d_adapter[t];
        right = past >= 0 && fresh >= 0 && (int64_t)past + fresh <= (int64_t)p.pages_per_seq * kv4::PAGE;
    }
    const int told = *p.d_n_free, n_free = min(max(told, 0), p.free_capacity);
    if ((t < B && !right) || told != n_free) atomicOr(err, LLAMA_DEVERR_INPUT);
    const int held = right ? (int)(((unsigned)past + kv4::PAGE - 1) / kv4::PAGE) : 0;
    int n = right ? fresh : 0;
    int need = right ? (int)(((unsigned)(past + fresh) + kv4::PAGE - 1) / kv4::PAGE) - held : 0;
    unsigned cn = (unsigned)n, cp = (unsigned)need;
    scan2(cn, cp, part);
    // both sums only grow, so the admitted requests are a prefix of the valid ones
    const bool ok = right && cn <= (unsigned)p.max_rows && cp <= (unsigned)n_free;
    if (ok) {
        atomicMax(&total_rows, (int)cn);
        atomicMax(&total_pages, (int)cp);
    } else {
        n = need = 0;
    }
    __syncthreads();
    const int rows = total_rows, pages = total_pages;
    const int end = min((int)cn, rows);
    if (t < B) {
        cu[t + 1] = end;
        page_end[t] = min((int)cp, pages);
        held_of[t] = held;
        n_new_s[t] = n;
        first[t] = past - (end - n);
        p.d_cu[t + 1] = end;
        p.d_kv_len[t] = right ? past + n : 0;
        p.d_admitted[t] = ok ? 1 : 0;
    }
    if (t == 0) {
        cu[0] = 0;
        p.d_cu[0] = 0;
    }
    if (A > 0) {
        // rows of each adapter: within a warp, requests of the same adapter find
        // each other; across warps their sums meet in a [warp][adapter] table
        const int lane = t & 31, warp = t >> 5;
        const int a = (t < B && n > 0 && adapter >= 0 && adapter < A) ? adapter : -1;
        const unsigned peers = __match_any_sync(0xffffffffu, a);
        __syncwarp();
        int before = 0, all = 0;
        if (a >= 0) {
            for (unsigned m = peers; m; m &= m - 1) {
                const int l = __ffs(m) - 1, v = n_new_s[warp * 32 + l];
                before += l < lane ? v : 0;
                all += v;
            }
            if (before == 0) dyn[warp * A + a] = all;      // the first of its peers (n > 0): one writer
        }
        __syncthreads();
        unsigned mine = 0, tiles = 0;
        if (t < A) {
            int sum = 0;
            for (int w = 0; w < warps; ++w) {
                const int v = dyn[w * A + t];
                dyn[w * A + t] = sum;
                sum += v;
            }
            mine = (unsigned)sum;
            tiles = (mine + LLAMA_LORA_TILE - 1) / LLAMA_LORA_TILE;
        }
        const int count = (int)mine;
        scan2(mine, tiles, part);
        if (t < A) {
            a_rows[t] = count;
            a_start[t] = (int)mine - count;
            a_tiles[t] = (int)tiles;             // inclusive
            if (t == A - 1) {
                total_lora = (int)mine;
                total_tiles = (int)tiles;
            }
        }
        __syncthreads();
        if (t < B) lora[t] = a >= 0 ? a_start[a] + dyn[warp * A + a] + before : -1;
        const int nt = min(total_tiles, p.max_tiles);
        for (int i = t; i < p.max_tiles; i += THREADS) {
            int4 tile = make_int4(-1, 0, 0, 0);
            if (i < nt) {
                const int ad = above(a_tiles, A, i);
                const int skip = (i - (ad ? a_tiles[ad - 1] : 0)) * LLAMA_LORA_TILE;
                tile = make_int4(ad, a_start[ad] + skip, min(a_rows[ad] - skip, LLAMA_LORA_TILE), 0);
            }
            reinterpret_cast<int4*>(p.d_lora_tiles)[i] = tile;
        }
        if (t == 0) *p.d_n_tiles = nt;
    }
    __syncthreads();
    // fresh pages, taken from the end of the free list in request order
    for (int i = t; i < pages; i += THREADS) {
        const int b = above(page_end, B, i);
        const int j = held_of[b] + i - (b ? page_end[b - 1] : 0);
        p.d_table[(int64_t)b * p.pages_per_seq + j] = p.d_free[n_free - 1 - i];
    }
    if (t == 0) *p.d_n_free_out = n_free - pages;      // may be d_n_free itself: read by every thread above
    if (fused) {
        __syncthreads();                               // the table's new entries
        for (int r = t; r < p.max_rows; r += THREADS) fill_row(p, cu, first, lora, r, rows, total_lora, err);
    } else {
        if (t < B) {
            p.d_work[2 + t] = first[t];
            p.d_work[2 + B + t] = A > 0 ? lora[t] : -1;
        }
        if (t == 0) {
            p.d_work[0] = rows;
            p.d_work[1] = total_lora;
        }
    }
}

constexpr int ROW_THREADS = 256;

__global__ void __launch_bounds__(ROW_THREADS) plan_rows_kernel(const __grid_constant__ llama_batch_plan p, int* err) {
    __shared__ int cu[THREADS + 1], first[THREADS], lora[THREADS];
    pdl_launch_dependents();
    pdl_wait();
    for (int i = threadIdx.x; i <= p.B; i += ROW_THREADS) cu[i] = p.d_cu[i];
    for (int i = threadIdx.x; i < p.B; i += ROW_THREADS) {
        first[i] = p.d_work[2 + i];
        lora[i] = p.d_work[2 + p.B + i];
    }
    const int rows = p.d_work[0], lora_rows = p.d_work[1];
    __syncthreads();
    for (int r = blockIdx.x * ROW_THREADS + threadIdx.x; r < p.max_rows; r += gridDim.x * ROW_THREADS)
        fill_row(p, cu, first, lora, r, rows, lora_rows, err);
}

}  // namespace

int launch_batch_plan(const llama_batch_plan& p, int* err, cudaStream_t st) {
    const int fused = p.max_rows <= FUSED_ROWS;
    const size_t smem = (size_t)((p.B + 31) / 32) * p.n_adapters * sizeof(int);    // 64 KB at the limits
    static PerDeviceOnce once;
    int rc = once_per_device(once, []() -> int {
        LLAMA_CUDA_TRY(cudaFuncSetAttribute(batch_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            WARPS * LLAMA_PLAN_MAX_ADAPTERS * (int)sizeof(int)));
        return (int)LLAMA_OK;
    });
    if (rc) return rc;
    launch_pdl(batch_plan_kernel, dim3(1), dim3(THREADS), smem, st, p, fused, err);
    LLAMA_LAUNCH_CHECK();
    if (!fused) {
        launch_pdl(plan_rows_kernel, dim3(ceil_div(p.max_rows, ROW_THREADS)), dim3(ROW_THREADS), 0, st, p, err);
        LLAMA_LAUNCH_CHECK();
    }
    return LLAMA_OK;
}
