// What the two kernels of a prompt pass in blocks share: the layout of the
// operands the first leaves for the second.
#pragma once

#include "stepq_serve.cuh"

namespace stepq {

constexpr int kC = kBlockTokens;
constexpr int kTileBytes = kC * kDK * 2;    // one binary16 half of a [64][128] operand
constexpr int kSquareBytes = kC * kC * 2 * 2;  // hi and lo of a [64][64] operand
// per block and head, for the state: -beta c_t times the unscale of the K rows, beta,
// unscale of the rows that make U (plain linear attention: what of each token
// is left at the block's end, times the unscale of its K row), kept share of S
constexpr int kStateFloats = 3 * kC + kDK;
constexpr int kOutFloats = 2 * kC;          // for the output: unscale of the Q rows times c_t, of the P rows

// Byte of element (row, col) of an operand tile [64][128] (two halves of 64
// columns) and of a [64][64] one: rows of 128 bytes whose 16-byte chunks are
// permuted by the row, the layout the tensor cores read and in which eight rows
// of one chunk lie in different banks.
__device__ __forceinline__ int square_at(int row, int col) { return row * 128 + (((col >> 3) ^ row) & 7) * 16 + (col & 7) * 2; }
__device__ __forceinline__ int tile_at(int row, int col) { return (col >> 6) * (kTileBytes / 2) + square_at(row, col & 63); }

// The scratch of a launch over `blocks` blocks.
struct Scratch {
    int heads_k;  // heads the K and Q tiles are made for
    int halves;   // binary16 halves of K and Q
    size_t k, q, k2, inv, p, sv, ov, total;
};

__host__ __device__ inline Scratch scratch_of(int variant, int dtype, int heads, int share, long long blocks)
{
    Scratch s;
    s.heads_k = variant == kKda ? heads : heads / share;
    s.halves = variant == kKda || dtype == kF32 ? 2 : 1;
    const size_t tiles = (size_t)blocks * s.heads_k * s.halves * kTileBytes, bh = (size_t)blocks * heads;
    size_t o = 0;
    s.k = o;   o += tiles;
    s.q = o;   o += tiles;
    s.k2 = o;  o += variant == kKda ? tiles : 0;
    s.inv = o; o += variant == kLinear ? 0 : bh * kSquareBytes;
    s.p = o;   o += bh * kSquareBytes;
    s.sv = o;  o += bh * kStateFloats * 4;
    s.ov = o;  o += bh * kOutFloats * 4;
    s.total = o;
    return s;
}

// The operands of n blocks from first_block on, into the scratch.
cudaError_t launch_block_tiles(const PromptArgs &a, int first_block, int n, const Scratch &sc, cudaStream_t s);

}  // namespace stepq
