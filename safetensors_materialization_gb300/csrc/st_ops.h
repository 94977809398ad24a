// st_ops.h -- the operators on materialized tensors (st_rms_norm,
// st_gated_act, st_linear): checked arguments and kernel launches.  Not part
// of the public ABI.
#pragma once

#include <cstdint>

#include "st_internal.h"

namespace stmat {

constexpr float kE4M3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: the smallest scale, so that 1 / scale is finite

// Checked by the C entry points: dtypes known, sizes in range, pointers
// aligned to their itemsize, rows, cols > 0.
st_status launch_rms_norm(const st_rms_norm_args &a, void *stream);
st_status launch_gated_act(const st_gated_act_args &a, void *stream);
// The same with a scale for every 128 columns: F8_E4M3 output, scales of its own.
st_status launch_rms_norm_blocks(const st_rms_norm_args &a, void *stream);
st_status launch_gated_act_blocks(const st_gated_act_args &a, void *stream);
// The current device, its SMs and its error word (kErrProduct).
st_status product_device(int *dev, int *sms, uint32_t **err);
// 2^-126 to the scales of rows without columns.
st_status launch_empty_rows(float *scales, int64_t rows, void *stream, const char *op);
// form: NULL, or a checked one.
st_status launch_linear(const st_linear_args &a, const st_linear_form *form, void *stream);
st_status check_linear_form(const st_linear_args &a, const st_linear_form &form);
st_linear_form choose_linear_form(const st_linear_args &a, int sms, int clusters_of_2, int clusters_of_4);
// Bytes of workspace the product needs (rows that TMA cannot read).
int64_t linear_workspace(const st_linear_args &a);

st_status launch_block_linear(const st_block_linear_args &a, const st_linear_form *form, void *stream);
st_status check_block_linear_form(const st_block_linear_args &a, const st_linear_form &form);
st_linear_form choose_block_linear_form(const st_block_linear_args &a, int sms);
int64_t block_linear_workspace(const st_block_linear_args &a);
st_status launch_moe(const st_moe_args &a, void *stream);
int64_t moe_workspace(const st_moe_args &a);

}  // namespace stmat
