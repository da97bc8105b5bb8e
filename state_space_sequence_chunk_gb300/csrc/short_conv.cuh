// short_conv.cuh -- shared declarations of the short convolution over packed rows (not part of the ABI).
#pragma once

#include "f32x2.cuh"

namespace ssd {

struct ShortConv {
    const int* cu;               // first token of each sequence [nseq + 1], or NULL: equal lengths L
    int nseq, T, L, D;
    int act;                     // ssd_act
    int64_t xs;                  // elements from one row of x to the next
    int64_t batch, nslots;       // single tokens
    const int* slots;
    const void *x, *init, *dout, *dfin;
    const float *w, *bias;
    void *out, *fin, *dx, *dinit, *cache;
    float *dw, *db, *part;
    int TT, tiles, items;        // tokens of a tile, tiles, tiles and sequences of their own
};

int short_conv_tile(int64_t T, int D, int W, int dtype, bool backward, int sms);
cudaError_t launch_short_conv_fwd(ShortConv& p, int W, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_short_conv_bwd(ShortConv& p, int W, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_short_conv_step(const ShortConv& p, int W, int dtype, cudaStream_t stream);

}  // namespace ssd
