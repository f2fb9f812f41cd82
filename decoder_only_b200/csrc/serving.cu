// Entry points of the serving operators (batch plan, 4-bit paged cache,
// adapters): argument checks, then the launchers.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... P>
bool aligned4(P... p) { return ((... | reinterpret_cast<uintptr_t>(p)) & 3u) == 0; }
bool known(int32_t dtype) { return dtype == LLAMA_F32 || dtype == LLAMA_BF16; }
int64_t per16(int32_t dtype) { return dtype == LLAMA_BF16 ? 8 : 4; }    // elements of 16 bytes
bool head_ok(int32_t hd) { return hd == 64 || hd == 128; }
constexpr int32_t MAX_HEADS = 65536;
constexpr int32_t MAX_PAGES = 0x7fffffff / kv4::PAGE;                   // slots are int32

bool store_ok(int32_t dtype, int32_t rows, int32_t n_kv, int32_t hd, int32_t n_pages) {
    if (!known(dtype) || rows < 0 || n_kv <= 0 || !head_ok(hd) || n_pages <= 0 || n_pages > MAX_PAGES) return false;
    return n_kv <= MAX_HEADS && (int64_t)rows * 2 * n_kv * (hd / 8) < 0x7fffff00;
}

}  // namespace

extern "C" {

int llama_op_batch_plan(const llama_batch_plan* plan, void* stream) {
    if (!plan) return LLAMA_ERR_INVALID_ARG;
    const llama_batch_plan& p = *plan;
    if (p.B <= 0 || p.B > LLAMA_PLAN_MAX_BATCH || p.pages_per_seq <= 0 || p.pages_per_seq > MAX_PAGES || p.n_pages <= 0 ||
        p.n_pages > MAX_PAGES || p.free_capacity < 0 || p.max_rows <= 0 || p.max_rows > (1 << 30) || p.n_adapters < 0 ||
        p.n_adapters > LLAMA_PLAN_MAX_ADAPTERS)
        return LLAMA_ERR_INVALID_ARG;
    if (!p.d_past || !p.d_new || !p.d_n_free || (p.free_capacity > 0 && !p.d_free) || !p.d_table || !p.d_cu || !p.d_kv_len ||
        !p.d_admitted || !p.d_n_free_out || !p.d_slots || !p.d_pos || !p.d_seq || !p.d_work)
        return LLAMA_ERR_INVALID_ARG;
    if (!aligned4(p.d_past, p.d_new, p.d_free, p.d_n_free, p.d_table, p.d_cu, p.d_kv_len, p.d_admitted, p.d_n_free_out, p.d_slots,
                  p.d_pos, p.d_seq, p.d_work, p.n_adapters > 0 ? p.d_adapter : nullptr, p.n_adapters > 0 ? p.d_lora_rows : nullptr,
                  p.n_adapters > 0 ? p.d_n_tiles : nullptr))
        return LLAMA_ERR_INVALID_ARG;
    const int64_t tiles = ((int64_t)p.max_rows + LLAMA_LORA_TILE - 1) / LLAMA_LORA_TILE + (p.B < p.n_adapters ? p.B : p.n_adapters);
    if (p.n_adapters > 0 && (!p.d_adapter || !p.d_lora_rows || !p.d_lora_tiles || !aligned16(p.d_lora_tiles) || !p.d_n_tiles ||
                             p.max_tiles < tiles))
        return LLAMA_ERR_INVALID_ARG;
    int* err = nullptr;
    int rc = op_error_word(&err);
    if (rc) return rc;
    return launch_batch_plan(p, err, (cudaStream_t)stream);
}

uint64_t llama_kv4_pool_bytes(int32_t n_pages, int32_t n_kv, int32_t head_dim) {
    if (n_pages <= 0 || n_pages > MAX_PAGES || n_kv <= 0 || n_kv > MAX_HEADS || !head_ok(head_dim)) return 0;
    return (uint64_t)n_pages * (uint64_t)n_kv * (uint64_t)kv4::head_bytes(head_dim);
}

int llama_op_kv4_append(int32_t dtype, const void* d_k, const void* d_v, const int32_t* d_slots, void* d_pool, int32_t rows,
                        int32_t n_kv, int32_t head_dim, int64_t k_stride, int64_t v_stride, int32_t n_pages, void* stream) {
    if (!store_ok(dtype, rows, n_kv, head_dim, n_pages)) return LLAMA_ERR_INVALID_ARG;
    if (rows == 0) return LLAMA_OK;
    if (!d_k || !d_v || !d_slots || !d_pool || !aligned16(d_k) || !aligned16(d_v) || !aligned16(d_pool) || !aligned4(d_slots))
        return LLAMA_ERR_INVALID_ARG;
    const int64_t width = (int64_t)n_kv * head_dim, unit = per16(dtype);
    if (k_stride < width || v_stride < width || k_stride % unit || v_stride % unit) return LLAMA_ERR_INVALID_ARG;
    int* err = nullptr;
    int rc = op_error_word(&err);
    if (rc) return rc;
    return launch_kv4_append(dtype, d_k, d_v, d_slots, static_cast<uint8_t*>(d_pool), rows, n_kv, head_dim, k_stride, v_stride,
                             (int64_t)n_pages * kv4::PAGE, err, (cudaStream_t)stream);
}

int llama_op_kv4_read(int32_t dtype, const void* d_pool, const int32_t* d_slots, void* d_k, void* d_v, int32_t rows, int32_t n_kv,
                      int32_t head_dim, int32_t n_pages, void* stream) {
    if (!store_ok(dtype, rows, n_kv, head_dim, n_pages)) return LLAMA_ERR_INVALID_ARG;
    if (rows == 0) return LLAMA_OK;
    if (!d_k || !d_v || !d_slots || !d_pool || !aligned16(d_k) || !aligned16(d_v) || !aligned16(d_pool) || !aligned4(d_slots))
        return LLAMA_ERR_INVALID_ARG;
    int* err = nullptr;
    int rc = op_error_word(&err);
    if (rc) return rc;
    const int64_t width = (int64_t)n_kv * head_dim;
    return launch_kv4_read(dtype, d_k, d_v, d_slots, static_cast<const uint8_t*>(d_pool), rows, n_kv, head_dim, width, width,
                           (int64_t)n_pages * kv4::PAGE, err, (cudaStream_t)stream);
}

uint64_t llama_op_attention_kv4_work_bytes(int32_t H, int32_t n_kv, int32_t head_dim, int32_t max_q) {
    if (H <= 0 || H > MAX_HEADS || n_kv <= 0 || H % n_kv || !head_ok(head_dim) || max_q <= 0) return 0;
    return attention_kv4_work_bytes(H, n_kv, head_dim, max_q);
}

int llama_op_attention_kv4(int32_t dtype, const void* d_q, int64_t q_stride, const void* d_pool, int32_t n_pages,
                           const int32_t* d_table, int32_t pages_per_seq, const int32_t* d_kv_len, const int32_t* d_cu,
                           int32_t max_q, void* d_o, int32_t B, int32_t rows, int32_t H, int32_t n_kv, int32_t head_dim,
                           void* d_work, uint64_t work_bytes, void* stream) {
    if (!known(dtype) || B <= 0 || B > LLAMA_PLAN_MAX_BATCH || rows < 0 || H <= 0 || n_kv <= 0 || H % n_kv || H > MAX_HEADS ||
        !head_ok(head_dim) || n_pages <= 0 || n_pages > MAX_PAGES || pages_per_seq <= 0 || pages_per_seq > MAX_PAGES ||
        max_q <= 0 || (int64_t)max_q * (H / n_kv) > (1 << 30))
        return LLAMA_ERR_INVALID_ARG;
    if (!d_cu && (rows != B || max_q != 1)) return LLAMA_ERR_INVALID_ARG;
    if (rows == 0) return LLAMA_OK;
    if (!d_q || !d_pool || !d_table || !d_kv_len || !d_o || !d_work || !aligned16(d_q) || !aligned16(d_pool) || !aligned16(d_o) ||
        !aligned16(d_work) || !aligned4(d_table, d_kv_len, d_cu) || q_stride < (int64_t)H * head_dim || q_stride % per16(dtype))
        return LLAMA_ERR_INVALID_ARG;
    if (work_bytes < attention_kv4_work_bytes(H, n_kv, head_dim, max_q)) return LLAMA_ERR_OOM;
    int* err = nullptr;
    int rc = op_error_word(&err);
    if (rc) return rc;
    return launch_attention_kv4(dtype, d_q, q_stride, static_cast<const uint8_t*>(d_pool), n_pages, d_table, pages_per_seq, d_kv_len,
                                d_cu, max_q, d_o, B, rows, H, n_kv, head_dim, static_cast<float*>(d_work), err,
                                (cudaStream_t)stream);
}

uint64_t llama_op_lora_work_bytes(int32_t rows, int32_t rank) {
    if (rows <= 0 || rank <= 0 || rank % 8 || rank > LLAMA_LORA_MAX_RANK) return 0;
    return lora_work_bytes(rows, rank);
}

int llama_op_lora(int32_t dtype, const void* d_x, int64_t ldx, const void* d_A, const void* d_B, const float* d_scale, float* d_y,
                  int64_t ldy, const int32_t* d_rows, const int32_t* d_tiles, const int32_t* d_n_tiles, int32_t max_tiles,
                  int32_t rows, int32_t d, int32_t n, int32_t rank, int32_t n_adapters, void* d_work, uint64_t work_bytes,
                  void* stream) {
    if (!known(dtype) || rows < 0 || d <= 0 || d % 8 || d > (1 << 24) || n <= 0 || n % 4 || n > (1 << 24) || rank <= 0 ||
        rank % 8 || rank > LLAMA_LORA_MAX_RANK || n_adapters <= 0 || max_tiles < 0 || max_tiles > 65535)
        return LLAMA_ERR_INVALID_ARG;
    if (rows == 0 || max_tiles == 0) return LLAMA_OK;
    if (!d_x || !d_A || !d_B || !d_scale || !d_y || !d_rows || !d_tiles || !d_n_tiles || !d_work) return LLAMA_ERR_INVALID_ARG;
    if (!aligned16(d_x) || !aligned16(d_A) || !aligned16(d_B) || !aligned16(d_y) || !aligned16(d_tiles) || !aligned4(d_scale, d_rows, d_n_tiles) ||
        !aligned16(d_work) || ldx < d || ldx % per16(dtype) || ldy < n || ldy % 4)
        return LLAMA_ERR_INVALID_ARG;
    if (work_bytes < lora_work_bytes(rows, rank)) return LLAMA_ERR_OOM;
    int* err = nullptr;
    int rc = op_error_word(&err);
    if (rc) return rc;
    return launch_lora(dtype, d_x, ldx, d_A, d_B, d_scale, d_y, ldy, d_rows, d_tiles, d_n_tiles, max_tiles, rows, d, n, rank,
                       n_adapters, static_cast<float*>(d_work), err, (cudaStream_t)stream);
}

}  // extern "C"
