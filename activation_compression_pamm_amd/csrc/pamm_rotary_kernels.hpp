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
    int num_cus;
    // how the work is cut: lanes of a row, tokens of a workgroup at a time, entries a token has in
    // the table, and workgroups that take the queries
    int lanes_log, T, width, blocks_q;
};

// Fills in how the work is cut; the number of workgroups.
int rotary_shape(RotaryArgs& a, int dtype, bool norm, bool backward);
hipError_t run_rotary(const RotaryArgs& a, int blocks, int dtype, hipStream_t st);
hipError_t run_rotary_backward(const RotaryArgs& a, int blocks, int dtype, hipStream_t st);

}  // namespace pamm
