// m2_chunk.hpp -- what the kernels of the chunked Mamba-2 mixer share: the
// record of a chunk's B and C, and how the work is divided.
#pragma once

#include "delta_chunk.hpp"
#include "kernels.hpp"

namespace selscan {
namespace m2chunk {

using namespace smm;
using dchunk::kC;
using dchunk::lds_barrier;
using dchunk::scalar;

constexpr int kBlock = 1024;   // bytes of an operand block: 16 bytes a lane

// Record of one (batch, chunk, group), in the order that lanes hold MFMA
// operands, so that a wave's load of an operand is 1 KB in a row.  NP: N rounded
// up to 32, 64 or 128; three bf16 planes each.
//   C [NP / 32][4][3]: rows 16 tt + i, k-step ks; lane 16 g + i has n = 32 ks +
//     4 g .. and 32 ks + 16 + 4 g .. (the order in which a state's C tiles hold n)
//   B [NP / 16][2][3]: its transpose, rows n = 16 nt + i; lane 16 g + i has
//     tokens 32 ks + 8 g ..
//   G [6][3] = C B^T on and below the diagonal, zero above: tiles (tt, ks) =
//     (0, 0), (1, 0), (2, 0), (2, 1), (3, 0), (3, 1); lane 16 g + i has row 16
//     tt + i, columns 32 ks + 8 g ..
template <int NP>
struct Rec {
    static constexpr int blocks = NP / 32 * 12;   // of C, and of B
    static constexpr int C = 0;
    static constexpr int B = blocks * kBlock;
    static constexpr int G = 2 * blocks * kBlock;
    static constexpr int bytes = G + 18 * kBlock;
};
__device__ __forceinline__ constexpr int g_tile(int tt, int ks) { return tt < 2 ? tt : 2 * tt - 2 + ks; }

__device__ __forceinline__ int64_t seq_len(const M2ConvArgs& a, int64_t b) {
    return a.conv.lengths ? min((int64_t)max(__builtin_amdgcn_readfirstlane(a.conv.lengths[b]), 0), a.L) : a.L;
}

// How the scan is divided: `units` of 16 ct value columns of a head share a
// group's records; `waves` of them are a workgroup, `sets` workgroups a group.
// A sequence's chunks are walked in segments at once, `all` for all sequences:
// `segs` of `per` chunks to a sequence, or (segs = 0) about `want` in all, cut
// from the sequences' lengths on the device.
struct Plan {
    int64_t chunks;
    int64_t all, segs, per, want;
    int ct, cols, units, waves, sets, np;
};

// Where the segments lie.  Cut on the device: a lane has the sequence of its
// number (a batch of 64 and fewer), at least one segment each, of two chunks
// and more: T chunks in E sequences make T / per + E / 2 segments on average,
// and T / per + batch at most.
struct Cut {
    int per, first, n;   // the lane's sequence: its first segment, its segments
    __device__ __forceinline__ Cut(const M2ConvArgs& a, const Plan& pl) {
        const int lane = threadIdx.x & 63;
        const bool live = lane < a.batch;
        const int chunks = live ? (int)((min((int64_t)max(a.conv.lengths[live ? lane : 0], 0), a.L) + kC - 1) / kC) : 0;
        int all = chunks;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) all += __shfl_xor(all, o, 64);
        const int want = (int)pl.want, fit = max(want - __popcll(__ballot(chunks > 0)) / 2, want / 2);
        per = max(2, (all + fit - 1) / fit);
        n = live ? max(1, (chunks + per - 1) / per) : 0;
        int upto = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o, 64);
            if (lane >= o) upto += v;
        }
        first = upto - n;
    }
};

}  // namespace m2chunk
}  // namespace selscan
