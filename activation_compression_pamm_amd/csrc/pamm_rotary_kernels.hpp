// pamm_rotary_kernels.hpp -- argument block and launchers of the kernels that
// norm and rotate queries and keys.  Host code validates everything first.
#pragma once
#include "pamm_block_kernels.hpp"

namespace pamm {

struct RotaryArgs {
    HeadsArg q, k, qo, ko, dq, dk;  // dq, dk: gradients of the results (backward)
    const double* inv_freq;
    const void* positions;
    int64_t psb, pss;        // elements
    const int32_t* offset;
    const char *wq, *wk;
    float* part;             // [blocks][D]: partial sums of the weights' gradients, queries' blocks first
    float *dwq, *dwk;
    int64_t tokens;          // batch * seq
    int S, Hq, Hk, D, R2;    // R2: rotated pairs of a row
    int positions_64, inverse, interleaved;
    float magnitude, eps;
    int lanes_log, tokens_log;  // lanes a row, tokens a workgroup at a time
    int num_cus;
    int blocks_q;            // backward: workgroups that take the queries
};

// Fills in how the work is cut.
void rotary_shape(RotaryArgs& a, int dtype, bool backward);
// Workgroups of the backward pass; fills in those for the queries.
int rotary_backward_blocks(RotaryArgs& a, int dtype);
hipError_t run_rotary(const RotaryArgs& a, int dtype, hipStream_t st);
hipError_t run_rotary_backward(RotaryArgs a, int dtype, hipStream_t st);

}  // namespace pamm
