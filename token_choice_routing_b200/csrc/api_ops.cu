// C ABI entry points of the slot-sorting and 8-bit checkpoint operators (declared in
// include/moe_null.h): host-side argument checks, then stream-ordered launches.
#include "rows.cuh"

#include <climits>

using namespace moe;

static inline cudaStream_t S(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
static inline uint32_t* status_word(void* p) { return static_cast<uint32_t*>(p); }

constexpr int kMaxSlots = 32;          // slots of a token: one lane each
constexpr int kMaxWidth = 1 << 30;     // columns of a row (column counters are 32-bit)
constexpr int kMaxSortExperts = 1024;  // two per thread of the smaller CTA in the sort's scan, ids of ten bits

static int check_slots(int32_t T, int32_t K) {
  if (T < 0 || K < 1) return MOE_ERR_INVALID_ARG;
  return (K > kMaxSlots || (long long)T * K >= (long long)INT_MAX) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

static int check_sort(int32_t T, int32_t K, int32_t N) {
  const int r = check_slots(T, K);
  if (r != MOE_OK) return r;
  if (N < 1) return MOE_ERR_INVALID_ARG;
  return N > kMaxSortExperts ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

static int check_rows(int32_t T, int32_t K, int64_t rows, int32_t d, int32_t dtype) {
  const int r = check_slots(T, K);
  if (r != MOE_OK) return r;
  if (rows < 0 || d < 1 || dtype_bytes(dtype) == 0) return MOE_ERR_INVALID_ARG;
  return d > kMaxWidth ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

static int check_block(int64_t rows, int64_t cols, int32_t dtype) {
  if (rows < 0 || cols < 1 || dtype_bytes(dtype) == 0) return MOE_ERR_INVALID_ARG;
  return (cols > kMaxWidth || rows > ((int64_t)1 << 60) / cols) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

extern "C" {

size_t moe_sort_workspace_bytes(int32_t T, int32_t K, int32_t N) {
  return check_sort(T, K, N) == MOE_OK ? sort_workspace_bytes(T, K, N) : 0;
}

int moe_sort_slots(int32_t T, int32_t K, int32_t N, const void* ids, int32_t id_bytes, int32_t* counts,
                   int32_t* offsets, int32_t* perm_tok, int32_t* slot_row, void* workspace, moe_stream_t stream) {
  const int r = check_sort(T, K, N);
  if (r != MOE_OK) return r;
  if (id_bytes != 4 && id_bytes != 8) return MOE_ERR_INVALID_ARG;
  if (!counts || !offsets || !workspace) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ids || !perm_tok || !slot_row)) return MOE_ERR_INVALID_ARG;
  return launch_sort_slots(T, K, N, ids, id_bytes, counts, offsets, perm_tok, slot_row, workspace, S(stream));
}

int moe_permute(int32_t T, int32_t K, int64_t rows, int32_t d, int32_t dtype, const void* x, int64_t ldx,
                const int32_t* slot_row, void* xs, int64_t ldxs, void* status, moe_stream_t stream) {
  const int r = check_rows(T, K, rows, d, dtype);
  if (r != MOE_OK) return r;
  if (T == 0) return MOE_OK;
  if (!x || !slot_row || (rows > 0 && !xs) || ldx < d || ldxs < d) return MOE_ERR_INVALID_ARG;
  if (rows == 0 && !status) return MOE_OK;  // nothing to write, nowhere to record a bad index
  return launch_spread(T, K, rows, d, dtype, x, ldx, nullptr, 0, nullptr, nullptr, slot_row, xs, ldxs, nullptr,
                       status_word(status), S(stream));
}

int moe_permute_backward(int32_t T, int32_t K, int64_t rows, int32_t d, int32_t dtype, const void* dxs, int64_t lddxs,
                         const int32_t* slot_row, const void* base, int64_t ldbase, void* dx, int64_t lddx,
                         void* status, moe_stream_t stream) {
  const int r = check_rows(T, K, rows, d, dtype);
  if (r != MOE_OK) return r;
  if (T == 0) return MOE_OK;
  if ((rows > 0 && !dxs) || !slot_row || !dx || lddxs < d || lddx < d || (base && ldbase < d))
    return MOE_ERR_INVALID_ARG;
  return launch_collect(T, K, rows, d, dtype, dxs, lddxs, nullptr, slot_row, base, ldbase, dx, lddx,
                        status_word(status), S(stream));
}

int moe_unpermute(int32_t T, int32_t K, int64_t rows, int32_t d, int32_t dtype, const void* ys, int64_t ldys,
                  const float* weights, const int32_t* slot_row, const void* base, int64_t ldbase, void* y,
                  int64_t ldy, void* status, moe_stream_t stream) {
  const int r = check_rows(T, K, rows, d, dtype);
  if (r != MOE_OK) return r;
  if (T == 0) return MOE_OK;
  if ((rows > 0 && !ys) || !weights || !slot_row || !y || ldys < d || ldy < d || (base && ldbase < d))
    return MOE_ERR_INVALID_ARG;
  return launch_collect(T, K, rows, d, dtype, ys, ldys, weights, slot_row, base, ldbase, y, ldy, status_word(status),
                        S(stream));
}

int moe_unpermute_backward(int32_t T, int32_t K, int64_t rows, int32_t d, int32_t dtype, const void* dy, int64_t lddy,
                           const void* ys, int64_t ldys, const float* weights, const int32_t* slot_row, void* dys,
                           int64_t lddys, float* dweights, void* status, moe_stream_t stream) {
  const int r = check_rows(T, K, rows, d, dtype);
  if (r != MOE_OK) return r;
  if (T == 0) return MOE_OK;
  if (!dy || !weights || !slot_row || lddy < d || (dys && lddys < d) || (ys && ldys < d)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && ((!dys && !dweights) || ((ys != nullptr) != (dweights != nullptr)))) return MOE_ERR_INVALID_ARG;
  if (rows == 0 && !dweights && !status) return MOE_OK;
  return launch_spread(T, K, rows, d, dtype, dy, lddy, ys, ldys, nullptr, weights, slot_row, dys, lddys, dweights,
                       status_word(status), S(stream));
}

int moe_unpermute_backward8(int32_t T, int32_t K, int64_t rows, int32_t d, int32_t dtype, const void* dy, int64_t lddy,
                            const int8_t* codes, const uint8_t* scales, const float* weights, const int32_t* slot_row,
                            void* dys, int64_t lddys, float* dweights, void* status, moe_stream_t stream) {
  const int r = check_rows(T, K, rows, d, dtype);
  if (r != MOE_OK) return r;
  if (T == 0) return MOE_OK;
  if (!dy || (rows > 0 && (!codes || !scales)) || !weights || !slot_row || !dweights || lddy < d ||
      (dys && lddys < d))
    return MOE_ERR_INVALID_ARG;
  return launch_spread(T, K, rows, d, dtype, dy, lddy, codes, d, scales, weights, slot_row, dys, lddys, dweights,
                       status_word(status), S(stream));
}

size_t moe_checkpoint8_scales(int64_t cols) { return cols < 1 ? 0 : (size_t)((cols + 31) / 32); }

int moe_checkpoint8(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx, const int32_t* rows_used,
                    int8_t* codes, uint8_t* scales, void* status, moe_stream_t stream) {
  const int r = check_block(rows, cols, dtype);
  if (r != MOE_OK) return r;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || ldx < cols) return MOE_ERR_INVALID_ARG;
  return launch_checkpoint8(rows, (int)cols, dtype, x, ldx, rows_used, codes, scales, status_word(status), S(stream));
}

int moe_restore8(int64_t rows, int64_t cols, int32_t dtype, const int8_t* codes, const uint8_t* scales,
                 const int32_t* rows_used, void* x, int64_t ldx, void* status, moe_stream_t stream) {
  const int r = check_block(rows, cols, dtype);
  if (r != MOE_OK) return r;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || ldx < cols) return MOE_ERR_INVALID_ARG;
  return launch_restore8(rows, (int)cols, dtype, codes, scales, rows_used, x, ldx, status_word(status), S(stream));
}

int moe_swiglu_backward8(int64_t rows, int64_t F, int32_t packed, int32_t dtype, const int8_t* codes,
                         const uint8_t* scales, const void* dh, int64_t lddh, const int32_t* rows_used, void* dz,
                         int64_t lddz, void* h, int64_t ldh, void* status, moe_stream_t stream) {
  if (F < 1 || (packed && F % 64 != 0)) return MOE_ERR_INVALID_ARG;
  if (F > kMaxWidth / 2) return MOE_ERR_UNSUPPORTED;
  const int r = check_block(rows, 2 * F, dtype);
  if (r != MOE_OK) return r;
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !dh || !dz || lddh < F || lddz < 2 * F || (h && ldh < F)) return MOE_ERR_INVALID_ARG;
  return launch_swiglu_backward8(rows, (int)F, packed, dtype, codes, scales, dh, lddh, rows_used, dz, lddz, h, ldh,
                                 status_word(status), S(stream));
}

}  // extern "C"
