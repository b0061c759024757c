// pamm_cache_kernels.hpp -- argument blocks and launchers of the kernels over
// a cache in 8 bits.  Host code validates everything first.
#pragma once
#include "pamm_block_kernels.hpp"

namespace pamm {

struct ScalesArg {
    float* p;
    int64_t sb, ss, sh;  // elements
};

// What the cache adds to AttnArgs, whose k and v are its 8-bit tensors.
struct Cache8Args {
    HeadsArg kt, vt;  // tails
    ScalesArg ks, vs;
    int block_log;
};

int attention8_splits(int64_t B, int64_t Sq, int64_t Sk, int64_t Hkv, int64_t G, bool lengths, int num_cus);
hipError_t run_attention8(const AttnArgs& a, const Cache8Args& c, int dtype, hipStream_t st);

struct AppendArgs {
    struct One {
        HeadsArg x, tail, to;  // new tokens, tail, 8 bits
        ScalesArg scale;
    } t[2];                    // keys, values
    const int32_t* new_len;
    int32_t* lengths;
    int B, n, room, Hkv, D, block_log;
    int touched;               // blocks that n tokens can touch
    int advance;
};
hipError_t run_cache8_append(const AppendArgs& a, int dtype, hipStream_t st);

}  // namespace pamm
