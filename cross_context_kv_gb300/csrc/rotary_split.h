// rotary_split.h -- how kvfix_rotary's work falls to threads: host arithmetic and a thread's place in
// it, without CUDA types, so that it can be checked at the ends of the documented sizes on a CPU.
#pragma once

#ifdef __CUDACC__
#define KVFIX_ON_BOTH __host__ __device__ __forceinline__
#else
#define KVFIX_ON_BOTH inline
#endif

namespace kvfix {

constexpr int kRotaryThreads = 256;

struct RotarySplit {
    int columns;      // threads per (token, run of heads)
    int runs;         // threads that share a token's heads
    int tile;         // tokens per block
    int tiles;        // blocks per (chunk, layers)
    int layer_block;  // layers per block
    int layer_blocks;
};

// The pairs of a column of half layouts whose halves no vector border meets.
KVFIX_ON_BOTH int mixed_pairs(int rotary_dim) { return rotary_dim % 8 == 0 ? 4 : rotary_dim % 4 == 0 ? 2 : 1; }

// The split.  A thread has a token's heads one after another, four in flight, while that leaves
// enough threads to fill the GPU; with fewer tokens the heads are spread over 2, 4, ... threads until
// each has one (8 x 512 tokens x 40 heads: 14.3 us, about twice that if spread four times as far).  Blocks take
// several layers (a thread's angles are used for all of them) where that leaves four blocks an SM.
// chunks * layers * tokens is below 2^31 (and so are the blocks); sums past a size are 64 bits wide.
inline RotarySplit rotary_split(int chunks, int layers, int tokens, int heads, int dim, int rotary_dim, bool half, bool in_place) {
    RotarySplit w;
    if (half && rotary_dim % 16 != 0) {
        const int P = mixed_pairs(rotary_dim), border = (rotary_dim + 7) / 8 * 8;
        w.columns = in_place ? rotary_dim / (2 * P) : border / (2 * P) + (dim - border) / 8;
    } else {
        w.columns = in_place ? (rotary_dim + 15) / 16 : dim / 16;
    }
    const int slots = kRotaryThreads / w.columns;
    const double rows = (double)chunks * layers * tokens, full = 152.0 * 1536.0;
    w.runs = 1;
    while (w.runs * 2 <= slots && w.runs < heads && rows * w.columns * w.runs < full) w.runs *= 2;
    w.tile = slots / w.runs;
    if (w.tile > tokens) w.tile = tokens;
    auto blocks = [](int n, int each) { return (int)(((long long)n + each - 1) / each); };
    w.tiles = blocks(tokens, w.tile);
    w.layer_block = 1;
    while (w.layer_block < 8 && w.layer_block * 2 <= layers &&
           (double)chunks * w.tiles * blocks(layers, 2 * w.layer_block) >= 4.0 * 152)
        w.layer_block *= 2;
    w.layer_blocks = blocks(layers, w.layer_block);
    return w;
}

// Where a thread of block `block` stands, where it has a token; the ends of a block's tokens and layers
// are taken without a sign or from the rest, as their sums may pass 2^31.
struct RotaryPlace {
    int column, run, chunk, layer0;
    unsigned token;
};
KVFIX_ON_BOTH bool rotary_place(const RotarySplit& w, int tokens, unsigned block, int thread, RotaryPlace& p) {
    const int slot = thread / w.columns;
    p.column = thread - slot * w.columns;
    const int in_tile = slot / w.runs;
    p.run = slot - in_tile * w.runs;
    p.layer0 = (int)(block % (unsigned)w.layer_blocks) * w.layer_block;
    block /= (unsigned)w.layer_blocks;
    p.chunk = (int)(block / (unsigned)w.tiles);
    p.token = (block - (unsigned)p.chunk * (unsigned)w.tiles) * (unsigned)w.tile + (unsigned)in_tile;
    return in_tile < w.tile && p.token < (unsigned)tokens;
}
KVFIX_ON_BOTH int rotary_layers(const RotarySplit& w, int layers, int layer0) {
    return layers - layer0 < w.layer_block ? layers - layer0 : w.layer_block;
}

}  // namespace kvfix
