// rotary.h -- the arguments of one kvfix_rotary call, as the kernel takes them.
#pragma once

#include "common.cuh"

namespace kvfix {

struct RotaryArgs {
    const uint16_t* in[2];  // queries, keys; a plane that is not given has no heads
    uint16_t* out[2];
    Plane ip[2], op[2];
    const int32_t* positions;  // [chunks][tokens]
    int chunks, layers, tokens, dim;
    int rotary_dim, layout;
    bool in_place;    // every plane: the values that do not rotate are where they belong
    float attention;  // factor of cos and sin
    // theta_i / 2 pi as a fraction of 2^64: a position times this, modulo 2^64, is the angle in
    // turns, exactly
    unsigned long long turns[kMaxHeadDim / 2];
};

// Fills rotary_dim, layout, attention and turns.
void rotary_angles(const kvfix_rope& rope, RotaryArgs* a);
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s);

}  // namespace kvfix
