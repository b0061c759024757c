// Sweeps the rule that cuts the work of norm and rotation into workgroups, as it
// is (its source is part of this one): what kernels put into LDS fits, both
// tensors get workgroups, and the stated workspace holds what is written.  Host code only.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "pamm_rotary.hip"
#include "pamm_rotary_api.hip"

#define CHECK(x) do { if (!(x)) { printf("%s:%d: %s (dtype %d, D %d, R2 %d, interleaved %d, heads %d/%d, tokens %lld)\n", \
    __FILE__, __LINE__, #x, dtype, D, R2, inter, Hq, Hk, (long long)tokens); exit(1); } } while (0)

static void shape(int dtype, int D, int R2, int inter, int Hq, int Hk, int64_t tokens, int cus) {
    using namespace pamm;
    RotaryArgs a;
    memset(&a, 0, sizeof a);
    a.tokens = tokens, a.S = (int)tokens, a.Hq = Hq, a.Hk = Hk, a.D = D, a.R2 = R2, a.interleaved = inter, a.num_cus = cus;
    for (int kind = 0; kind < 3; ++kind) {  // rotation, norm and rotation, its backward pass
        RotaryArgs r = a;
        const int blocks = rotary_shape(r, dtype, kind > 0, kind == 2);
        const int P = dtype == DT_BF16 ? 8 : 4, lanes = 1 << r.lanes_log, groups = kThreads / lanes, pairs = pairs_of(r, dtype);
        CHECK(2 * lanes * P >= D && lanes <= 16);
        CHECK(r.T >= 1 && r.T <= kTokens && r.T * r.width <= kTablePairs);
        // the last entry that a lane reads of a token's angles
        CHECK(pairs == PAIRS_HALF ? r.width >= R2 + P : pairs == PAIRS_INTER ? r.width >= lanes * P : r.width >= R2 + 1);
        const int heads = Hq > Hk ? Hq : Hk;
        CHECK(r.T == 1 || (int64_t)r.T * heads <= 1 << 20);
        CHECK(kind != 0 || groups % r.T == 0);
        CHECK(blocks >= r.blocks_q && (int64_t)r.blocks_q * kThreads < (int64_t)1 << 32 && (int64_t)blocks * kThreads < (int64_t)1 << 32);
        if (tokens > 0) CHECK(r.blocks_q >= 1 && (Hk == 0 || blocks > r.blocks_q));
    }
    // the stated workspace is what the backward pass writes a row a workgroup to
    RotaryArgs r = a;
    r.num_cus = num_cus();
    const int blocks = rotary_shape(r, dtype, true, true);
    pamm_rotary_t p;
    memset(&p, 0, sizeof p);
    p.dtype = dtype, p.interleaved = inter, p.batch = 1, p.seq = tokens, p.heads_q = Hq, p.heads_k = Hk, p.head_dim = D;
    p.rot_dim = 2 * R2, p.magnitude = 1.0f;
    CHECK(pamm_rotary_backward_workspace_size(&p) >= (size_t)blocks * D * sizeof(float));
}

int main() {
    static const int heads[][2] = {{1, 0}, {1, 1}, {12, 12}, {32, 8}, {8, 32}, {333, 1}, {70000, 70000}, {1 << 28, 1}};
    static const int64_t tokens[] = {0, 1, 2, 63, 511, 512, 513, 8192, 20547, 100000, 2147483647LL};
    for (int dtype = 0; dtype < 2; ++dtype)
        for (int D = dtype ? 8 : 4; D <= PAMM_MAX_HEAD_DIM; D += dtype ? 8 : 4)
            for (int R2 = 0; 2 * R2 <= D; ++R2)
                for (int inter = 0; inter < 2; ++inter)
                    for (auto& h : heads)
                        for (int64_t t : tokens)
                            for (int cus : {1, 64, 256, 304}) shape(dtype, D, R2, inter, h[0], h[1], t, cus);
    printf("shape driver ok\n");
    return 0;
}
