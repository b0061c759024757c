// pamm_block_kernels.hpp -- argument blocks and launchers of the kernels
// around the projection (attention, RMS norm, gradient clipping).  Host code
// validates everything before calling a launcher; launchers only enqueue work
// on the given stream and report hipGetLastError().
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pamm {

// A [batch x sequence x heads x dim] tensor; strides in bytes.
struct HeadsArg {
    char* p;
    int64_t sb, ss, sh;
};

struct AttnArgs {
    HeadsArg q, k, v, o, dout, dq, dk, dv;
    float* lse;             // [B x H x Sq]
    float* delta;           // [B x H x Sq]: <do, o>, backward only
    const int32_t* q_len;   // [B] or null
    const int32_t* kv_len;  // [B] or null
    int B, Sq, Sk, H, Hkv, G, D;  // G = H / Hkv
    int causal;
    int window;             // 0: none
    bool hides;             // the mask may hide a key between those of a block that are seen: waves mark
                            // what they have to leave to the second kernel, and it is launched
    float scale;
    int nsplit;             // parts of the key axis (forward)
    float* part_o;          // [B x H x Sq x nsplit x D] when nsplit > 1
    float* part_lse;        // [B x H x Sq x nsplit], log2 units
    int nsplit_kv;          // parts of the query axis (dk and dv)
    float* part_dk;         // [nsplit_kv x B x Hkv x Sk x D] when nsplit_kv > 1
    float* part_dv;
    int32_t* marks;         // [dq items, dk/dv items][4 waves]: 1 if it has to be computed again
    int dq_items;
    int num_cus;
};

// Rows (queries x heads that share a key/value head) up to which the forward
// kernel gives each wave keys of its own instead of rows of its own.
constexpr int kFewRows = 32;

// Parts into which the forward pass cuts the key axis, at most kMaxSplits.
constexpr int kMaxSplits = 64;
int attention_splits(int64_t B, int64_t Sq, int64_t Sk, int64_t Hkv, int64_t G, bool lengths, int num_cus);
// Parts into which the dk/dv pass cuts the queries of a key tile.
int attention_dkv_splits(int64_t B, int64_t Sq, int64_t Sk, int64_t Hkv, int64_t G, int dtype, int num_cus);
hipError_t run_attention(const AttnArgs& a, int dtype, hipStream_t st);
hipError_t run_attention_backward(const AttnArgs& a, int dtype, hipStream_t st);

// Longest row of the RMS norm in 16-byte vectors: 1024 threads hold it in
// registers, four vectors each.
constexpr int64_t kMaxNormVectors = 4096;

struct NormArgs {
    const char *x, *r, *w, *dy, *dh;
    char *h, *y, *dx;
    uint8_t* q;
    float *qscale, *rstd, *dw;
    float* part;  // [blocks x d] partial sums of dw
    int64_t ldx, ldr, ldh, ldy, ldq, lddy, lddh, lddx;  // bytes
    int64_t n;
    int d;
    float eps;
    int num_cus;
};

hipError_t run_add_rms_norm(const NormArgs& a, int dtype, hipStream_t st);
// Workgroups of the backward pass, each of which leaves one row of partial sums.
int norm_backward_blocks(int64_t n, int64_t d, int dtype, int num_cus);
hipError_t run_add_rms_norm_backward(const NormArgs& a, int dtype, hipStream_t st);

// Tensors one launch of the clipping kernels covers (their descriptors travel
// as kernel arguments), and workgroups of one launch.
constexpr int kClipTensors = 60;
constexpr int kClipBlocks = 1024;

struct ClipTensor {
    const char* data;
    char* out;
    int64_t cols, rows, ld, ld_out;  // elements
    int32_t dtype, out_dtype;
    int64_t first_chunk;             // of this launch
};
struct ClipArgs {
    ClipTensor t[kClipTensors];
    int count;
    int parts;        // partial sums of this launch (forward) or of all (scaling)
    int64_t chunks;   // of this launch
    int in_place;     // every output of the call is its input
    double* part;
    float* norm;
    float max_norm, eps;
};

int64_t clip_chunks(const ClipTensor& t);
hipError_t run_clip_sum(const ClipArgs& a, hipStream_t st);
hipError_t run_clip_scale(const ClipArgs& a, bool write, hipStream_t st);

}  // namespace pamm
