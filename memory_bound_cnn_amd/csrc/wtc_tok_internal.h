// Internal declarations of the token operators (include/wtconv_tokens.h): the
// launchers that wtconv_tok_api.cpp calls after its checks, and the launch
// shapes that the checks and the kernels share.  Not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/wtconv_tokens.h"

namespace wtc {

// Root-mean-square norm: workgroups of the backward pass, each with one record
// of C partial sums of dw (four workgroups of 256 threads per compute unit).
constexpr int kRmsMaxParts = 1024;
int rms_backward_parts(const wtc_rms_desc* d);
int launch_rms_forward(const wtc_rms_desc* d, const void* x, const void* r, const float* w, void* y, void* h,
                       float* rstd, float* scale, void* stream);
int launch_rms_backward(const wtc_rms_desc* d, const void* dy, const void* dh, const void* h, const float* w,
                        const float* rstd, void* dx, float* dw, float* parts, void* stream);

int launch_rotary(const wtc_rotary_desc* d, const void* x, const int* pos, const float* inv_freq, void* y,
                  void* stream);

// least: an element is kept where its 16 bits are at least this; 65536 drops all
int launch_dropout(long long n, int dtype, unsigned least, const void* x, const void* r,
                   const unsigned long long* rng, void* y, void* stream);

// workspaces: the splits' partial results; backward also rowsum(dout * out) [Hq, T]
size_t attn_forward_bytes(const wtc_attn_desc* d);
size_t attn_backward_bytes(const wtc_attn_desc* d);
int launch_attn_forward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const int* cu, void* out,
                        float* lse, void* out_low, void* workspace, void* stream);
int launch_attn_backward(const wtc_attn_desc* d, const void* q, const void* k, const void* v, const void* out,
                         const float* lse, const void* out_low, const void* dout, const int* cu, void* dq, void* dk, void* dv,
                         void* workspace, void* stream);

int layer_backward_parts(const wtc_layer_desc* d);
int launch_layer_forward(const wtc_layer_desc* d, const void* x, const void* r, const float* w, const float* b, void* y,
                         void* h, float* stats, void* stream);
int launch_layer_backward(const wtc_layer_desc* d, const void* dy, const void* dh, const void* h, const float* w,
                          const float* stats, void* dx, float* dw, float* db, float* parts, void* stream);

// Gated recurrence: the forward pass keeps the state before every kScanKept-th token for the backward pass
constexpr int kScanKept = 8;
size_t scan_workspace(const wtc_scan_desc* d);
int launch_scan_forward(const wtc_scan_desc* d, const void* x, const void* f, const int* cu, const float* state, void* y,
                        float* last, float* kept, void* workspace, void* stream);
int launch_scan_backward(const wtc_scan_desc* d, const void* x, const void* f, const int* cu, const float* state,
                         const float* kept, const void* dy, const float* dlast, void* dx, void* df, float* dstate,
                         void* workspace, void* stream);
int launch_scan_step(const wtc_scan_desc* d, const void* x, const void* f, const float* state, void* y, float* out,
                     void* stream);

size_t order_workspace(long long n, int E);
int launch_expert_order(long long n, int E, const int* experts, int* slot, int* pair, int* cu, void* workspace, void* stream);
int launch_rows_gather(const wtc_rows_desc* d, const void* x, const int* slot, const int* cu, void* rows, void* stream);
int launch_rows_sum(const wtc_rows_desc* d, const void* rows, const float* weights, const int* slot, void* y, void* stream);
int launch_rows_sum_backward(const wtc_rows_desc* d, const void* dy, const void* rows, const float* weights, const int* slot,
                             const int* cu, void* drows, float* dweights, void* stream);

size_t expert_weights_workspace(const wtc_expert_desc* d);
int launch_expert_forward(const wtc_expert_desc* d, const void* x, const void* w, const void* b, const int* cu, void* y,
                          void* stream);
int launch_expert_input_grad(const wtc_expert_desc* d, const void* dy, const void* w, const int* cu, void* dx, void* stream);
int launch_expert_weight_grad(const wtc_expert_desc* d, const void* dy, const void* x, const int* cu, void* dw, void* db,
                              void* workspace, void* stream);

}  // namespace wtc
