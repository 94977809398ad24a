// st_ops.cpp -- C entry points of the operators on materialized tensors:
// argument checks; the kernels are in st_rowops.cu and st_linear.cu.
#include <cstdint>

#include "st_ops.h"

using namespace stmat;

namespace {

// One grid dimension of rows, and tile coordinates that stay in 32 bits.
constexpr int64_t kMaxRows = 0x7fffff00;
constexpr int64_t kMaxCols = 0x7fffff00;

bool is_float16or32(st_dtype d) { return d == ST_BF16 || d == ST_F16 || d == ST_F32; }

// A [rows, cols] operand: NULL only when it may be absent; ld elements
// between rows (0: one row for all, inputs only), rows inside 63 bits.
st_status check_matrix(const char *op, const char *name, const void *p, int64_t ld, st_dtype dtype, int64_t rows,
                       int64_t cols, bool input) {
  if (!p) return set_error(ST_E_INVAL, "%s: %s is NULL", op, name);
  const int64_t item = static_cast<int64_t>(st_dtype_size(dtype));
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(item))
    return set_error(ST_E_ALIGN, "%s: %s is not aligned to its %lld-byte items", op, name, (long long)item);
  if (ld < cols && rows > 1 && !(input && ld == 0))
    return set_error(ST_E_INVAL, "%s: %s has %lld elements between rows of %lld", op, name, (long long)ld,
                     (long long)cols);
  int64_t span = 0;
  if (ld < 0 || __builtin_mul_overflow(ld, rows, &span) || __builtin_add_overflow(span, cols, &span) ||
      __builtin_mul_overflow(span, item, &span))
    return set_error(ST_E_INVAL, "%s: %s with %lld rows of stride %lld overflows 63 bits", op, name, (long long)rows,
                     (long long)ld);
  return ST_OK;
}

st_status check_vector(const char *op, const char *name, const void *p, st_dtype dtype) {
  const size_t item = st_dtype_size(dtype);
  if (reinterpret_cast<uintptr_t>(p) % item)
    return set_error(ST_E_ALIGN, "%s: %s is not aligned to its %zu-byte items", op, name, item);
  return ST_OK;
}

st_status check_sizes(const char *op, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxCols)
    return set_error(ST_E_INVAL, "%s: %lld x %lld is out of range (0 .. 2^31 - 256)", op, (long long)rows,
                     (long long)cols);
  return ST_OK;
}

// The output's dtype and, for 8 bits, exactly one of a given scale and an
// array for the rows' scales (no rows: which may be NULL).
st_status check_output(const char *op, st_dtype y, const float *scale, const float *scales, int64_t rows) {
  if (!is_float16or32(y) && y != ST_F8_E4M3)
    return set_error(ST_E_DTYPE, "%s: the output is BF16, F16, F32 or F8_E4M3, not %d", op, static_cast<int>(y));
  if (y == ST_F8_E4M3 ? (scale && scales) || (rows > 0 && !scale && !scales) : (scale || scales))
    return set_error(ST_E_INVAL, "%s: an F8_E4M3 output takes either scale or scales, another output neither", op);
  st_status s = check_vector(op, "scale", scale, ST_F32);
  return s != ST_OK ? s : check_vector(op, "scales", scales, ST_F32);
}

// The bytes of an operand: rows of `row` bytes, `pitch` apart.
struct Bytes {
  uintptr_t p;
  int64_t rows, pitch, row;
  uintptr_t end() const { return p + static_cast<uintptr_t>((rows - 1) * pitch + row); }
};

Bytes matrix_bytes(const void *p, int64_t ld, st_dtype dtype, int64_t rows, int64_t cols) {
  const int64_t item = static_cast<int64_t>(st_dtype_size(dtype));
  if (rows == 1 || ld == 0) return {reinterpret_cast<uintptr_t>(p), 1, 0, cols * item};
  if (ld == cols) return {reinterpret_cast<uintptr_t>(p), 1, 0, rows * cols * item};
  return {reinterpret_cast<uintptr_t>(p), rows, ld * item, cols * item};
}
Bytes array_bytes(const void *p, uint64_t bytes) { return {reinterpret_cast<uintptr_t>(p), 1, 0, static_cast<int64_t>(bytes)}; }

// Whether they share a byte.  Column ranges of one buffer interleave without.
bool overlap(const Bytes &a, const Bytes &b) {
  if (a.end() <= b.p || b.end() <= a.p) return false;
  if (a.rows > 1 && b.rows > 1 && a.pitch == b.pitch) {
    // Where b's rows start between two of a's; the ranges meet, so some pair
    // of rows is next to each other.
    const int64_t d = b.p >= a.p ? static_cast<int64_t>((b.p - a.p) % static_cast<uintptr_t>(a.pitch))
                                 : (a.pitch - static_cast<int64_t>((a.p - b.p) % static_cast<uintptr_t>(a.pitch))) % a.pitch;
    return d < a.row || d > a.pitch - b.row;
  }
  const Bytes &few = a.rows <= b.rows ? a : b, &many = a.rows <= b.rows ? b : a;
  for (int64_t i = 0; i < few.rows; ++i) {
    const uintptr_t from = few.p + static_cast<uintptr_t>(i * few.pitch), to = from + static_cast<uintptr_t>(few.row);
    // The first of the other's rows that ends beyond `from`.
    const uintptr_t first_end = many.p + static_cast<uintptr_t>(many.row);
    const int64_t j = first_end > from ? 0 : many.pitch ? static_cast<int64_t>((from - first_end) / static_cast<uintptr_t>(many.pitch)) + 1 : many.rows;
    if (j < many.rows && many.p + static_cast<uintptr_t>(j * many.pitch) < to) return true;
  }
  return false;
}

#define ST_TRY(expr)                         \
  do {                                       \
    const st_status try_status = (expr);     \
    if (try_status != ST_OK) return try_status; \
  } while (0)

st_status check_linear(const st_linear_args *a, bool *empty) {
  const char *op = "st_linear";
  ST_TRY(check_sizes(op, a->m, a->n));
  ST_TRY(check_sizes(op, a->m, a->k));
  const bool sixteen = (a->x_dtype == ST_BF16 || a->x_dtype == ST_F16) && a->w_dtype == a->x_dtype;
  const bool eight = a->x_dtype == ST_F8_E4M3 && (a->w_dtype == ST_F8_E4M3 || a->w_dtype == ST_F8_E5M2);
  if (!sixteen && !eight)
    return set_error(ST_E_DTYPE, "%s: x and weight are both BF16, both F16, or F8_E4M3 with F8_E4M3 or F8_E5M2 (got %d, %d)",
                     op, (int)a->x_dtype, (int)a->w_dtype);
  if (!is_float16or32(a->y_dtype)) return set_error(ST_E_DTYPE, "%s: the output is BF16, F16 or F32, not %d", op, (int)a->y_dtype);
  if (a->bias && !is_float16or32(a->bias_dtype))
    return set_error(ST_E_DTYPE, "%s: bias is BF16, F16 or F32, not %d", op, (int)a->bias_dtype);
  if (a->act < ST_ACT_NONE || a->act > ST_ACT_GELU_TANH) return set_error(ST_E_INVAL, "%s: unknown activation %d", op, (int)a->act);
  if (a->x_scale && a->x_scale_count != 1 && a->x_scale_count != a->m)
    return set_error(ST_E_INVAL, "%s: %lld scales for x (1 or m = %lld)", op, (long long)a->x_scale_count, (long long)a->m);
  if (a->w_scale && a->w_scale_count != 1 && a->w_scale_count != a->n)
    return set_error(ST_E_INVAL, "%s: %lld scales for weight (1 or n = %lld)", op, (long long)a->w_scale_count, (long long)a->n);
  ST_TRY(check_vector(op, "x_scale", a->x_scale, ST_F32));
  ST_TRY(check_vector(op, "w_scale", a->w_scale, ST_F32));
  *empty = a->m == 0 || a->n == 0;
  if (*empty) return ST_OK;
  if (a->k > 0) {
    ST_TRY(check_matrix(op, "x", a->x, a->ldx, a->x_dtype, a->m, a->k, true));
    ST_TRY(check_matrix(op, "weight", a->w, a->ldw, a->w_dtype, a->n, a->k, true));
  }
  if (a->bias) ST_TRY(check_vector(op, "bias", a->bias, a->bias_dtype));
  if (a->residual) ST_TRY(check_matrix(op, "residual", a->residual, a->ldr, a->y_dtype, a->m, a->n, true));
  ST_TRY(check_matrix(op, "y", a->y, a->ldy, a->y_dtype, a->m, a->n, false));
  // Other tiles still read x, the weight and the vectors while the first are
  // written; a residual's element is read by the thread that writes it in y.
  const Bytes y = matrix_bytes(a->y, a->ldy, a->y_dtype, a->m, a->n);
  auto apart = [&](const char *name, const Bytes &b) {
    return overlap(y, b) ? set_error(ST_E_INVAL, "%s: y overlaps %s (it may be the residual, the very matrix, and no other operand)", op, name) : ST_OK;
  };
  if (a->k > 0) {
    ST_TRY(apart("x", matrix_bytes(a->x, a->ldx, a->x_dtype, a->m, a->k)));
    ST_TRY(apart("weight", matrix_bytes(a->w, a->ldw, a->w_dtype, a->n, a->k)));
  }
  if (a->x_scale) ST_TRY(apart("x_scale", array_bytes(a->x_scale, 4 * a->x_scale_count)));
  if (a->w_scale) ST_TRY(apart("w_scale", array_bytes(a->w_scale, 4 * a->w_scale_count)));
  if (a->bias) ST_TRY(apart("bias", array_bytes(a->bias, a->n * st_dtype_size(a->bias_dtype))));
  if (a->residual && !(a->residual == a->y && (a->m == 1 || a->ldr == a->ldy)))
    ST_TRY(apart("the residual in part", matrix_bytes(a->residual, a->ldr, a->y_dtype, a->m, a->n)));
  return ST_OK;
}

st_status run_linear(const st_linear_args *a, const st_linear_form *form, void *stream) {
  if (!a) return set_error(ST_E_INVAL, "st_linear: NULL arguments");
  bool empty = false;
  ST_TRY(check_linear(a, &empty));
  if (empty) return ST_OK;
  if (form) ST_TRY(check_linear_form(*a, *form));
  const int64_t need = linear_workspace(*a);
  if (need && (!a->workspace || a->workspace_bytes < static_cast<uint64_t>(need)))
    return set_error(ST_E_INVAL, "st_linear: rows that are no multiples of 16 bytes apart need a workspace of %lld bytes, %llu given",
                     (long long)need, (unsigned long long)(a->workspace ? a->workspace_bytes : 0));
  if (need && reinterpret_cast<uintptr_t>(a->workspace) % 16)
    return set_error(ST_E_ALIGN, "st_linear: the workspace is not 16-byte aligned");
  if (need) {
    const Bytes space = array_bytes(a->workspace, static_cast<uint64_t>(need));
    if (overlap(space, matrix_bytes(a->y, a->ldy, a->y_dtype, a->m, a->n)) ||
        overlap(space, matrix_bytes(a->x, a->ldx, a->x_dtype, a->m, a->k)) ||
        overlap(space, matrix_bytes(a->w, a->ldw, a->w_dtype, a->n, a->k)) ||
        (a->residual && overlap(space, matrix_bytes(a->residual, a->ldr, a->y_dtype, a->m, a->n))))
      return set_error(ST_E_INVAL, "st_linear: the workspace overlaps an operand");
  }
  return launch_linear(*a, form, stream);
}

}  // namespace

extern "C" {

st_status st_rms_norm(const st_rms_norm_args *a, void *stream) {
  if (!a) return set_error(ST_E_INVAL, "st_rms_norm: NULL arguments");
  const char *op = "st_rms_norm";
  ST_TRY(check_sizes(op, a->rows, a->cols));
  if (!is_float16or32(a->x_dtype)) return set_error(ST_E_DTYPE, "%s: x is BF16, F16 or F32, not %d", op, (int)a->x_dtype);
  if (a->weight && !is_float16or32(a->w_dtype))
    return set_error(ST_E_DTYPE, "%s: weight is BF16, F16 or F32, not %d", op, (int)a->w_dtype);
  if (!(a->eps >= 0.0f)) return set_error(ST_E_INVAL, "%s: eps %g is not a non-negative number", op, (double)a->eps);
  if (a->h && !a->residual) return set_error(ST_E_INVAL, "%s: h without a residual", op);
  ST_TRY(check_output(op, a->y_dtype, a->scale, a->scales, a->rows));
  if (a->rows == 0) return ST_OK;
  if (a->cols == 0) return a->scales ? launch_empty_rows(a->scales, a->rows, stream, op) : ST_OK;
  ST_TRY(check_matrix(op, "x", a->x, a->ldx, a->x_dtype, a->rows, a->cols, true));
  if (a->residual) ST_TRY(check_matrix(op, "residual", a->residual, a->ldr, a->x_dtype, a->rows, a->cols, true));
  if (a->weight) ST_TRY(check_vector(op, "weight", a->weight, a->w_dtype));
  if (a->h) ST_TRY(check_matrix(op, "h", a->h, a->ldh, a->x_dtype, a->rows, a->cols, false));
  ST_TRY(check_matrix(op, "y", a->y, a->ldy, a->y_dtype, a->rows, a->cols, false));
  return launch_rms_norm(*a, stream);
}

st_status st_gated_act(const st_gated_act_args *a, void *stream) {
  if (!a) return set_error(ST_E_INVAL, "st_gated_act: NULL arguments");
  const char *op = "st_gated_act";
  ST_TRY(check_sizes(op, a->rows, a->cols));
  if (!is_float16or32(a->x_dtype)) return set_error(ST_E_DTYPE, "%s: gate is BF16, F16 or F32, not %d", op, (int)a->x_dtype);
  if (a->act < ST_ACT_NONE || a->act > ST_ACT_GELU_TANH) return set_error(ST_E_INVAL, "%s: unknown activation %d", op, (int)a->act);
  ST_TRY(check_output(op, a->y_dtype, a->scale, a->scales, a->rows));
  if (a->rows == 0) return ST_OK;
  if (a->cols == 0) return a->scales ? launch_empty_rows(a->scales, a->rows, stream, op) : ST_OK;
  ST_TRY(check_matrix(op, "gate", a->gate, a->ldg, a->x_dtype, a->rows, a->cols, true));
  if (a->up) ST_TRY(check_matrix(op, "up", a->up, a->ldu, a->x_dtype, a->rows, a->cols, true));
  ST_TRY(check_matrix(op, "y", a->y, a->ldy, a->y_dtype, a->rows, a->cols, false));
  return launch_gated_act(*a, stream);
}

st_status st_linear_workspace(const st_linear_args *a, uint64_t *bytes) {
  if (!a || !bytes) return set_error(ST_E_INVAL, "st_linear_workspace: NULL argument");
  bool empty = false;
  ST_TRY(check_linear(a, &empty));
  *bytes = empty ? 0 : static_cast<uint64_t>(linear_workspace(*a));
  return ST_OK;
}

st_status st_linear_choose(const st_linear_args *a, int32_t sms, int32_t clusters_of_2, int32_t clusters_of_4, st_linear_form *form) {
  if (!a || !form) return set_error(ST_E_INVAL, "st_linear_choose: NULL argument");
  if (sms < 2 || clusters_of_2 < 0 || clusters_of_4 < 0)
    return set_error(ST_E_INVAL, "st_linear_choose: no device has %d SMs and %d, %d clusters", sms, clusters_of_2, clusters_of_4);
  bool empty = false;
  ST_TRY(check_linear(a, &empty));
  if (empty) return set_error(ST_E_INVAL, "st_linear_choose: a product without rows or columns is not launched");
  *form = choose_linear_form(*a, sms, clusters_of_2, clusters_of_4);
  return ST_OK;
}

st_status st_linear(const st_linear_args *a, void *stream) { return run_linear(a, nullptr, stream); }

st_status st_linear_as(const st_linear_args *a, const st_linear_form *form, void *stream) {
  if (!form) return set_error(ST_E_INVAL, "st_linear_as: NULL form");
  return run_linear(a, form, stream);
}

}  // extern "C"
