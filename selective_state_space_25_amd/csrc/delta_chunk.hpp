// delta_chunk.hpp -- what the chunked gated delta rule's kernels share: the
// per-chunk record, bounded loads of 64-token pieces, operands in LDS.
#pragma once

#include "io.hpp"
#include "kernels.hpp"
#include "split_mfma.hpp"

namespace selscan {
namespace dchunk {

using namespace smm;

constexpr int kC = 64;             // tokens per chunk
constexpr int kBlocks = 10;        // 16 x 16 blocks on and below a chunk matrix's diagonal

// Record of one (batch, head, chunk), byte offsets.  T in three bf16 planes,
// each 10 row-major 16 x 16 blocks (block (t, s) at t (t + 1) / 2 + s); A the
// same; then per token e^cum, e^(last - cum), beta (zero past the sequence's
// end) and cum itself as doubles.  For the gradients A is fp32, and T's and
// A's blocks follow in three planes, each block transposed.
constexpr int kPlane = kBlocks * 512;
template <bool GRAD>
struct Rec {
    static constexpr int T = 0;
    static constexpr int A = 3 * kPlane;
    static constexpr int gam = A + (GRAD ? 2 : 3) * kPlane;   // (fp32 takes the place of two planes)
    static constexpr int tail = gam + 4 * kC;
    static constexpr int beta = tail + 4 * kC;
    static constexpr int cum = beta + 4 * kC;
    static constexpr int Tt = cum + 8 * kC;
    static constexpr int At = Tt + 3 * kPlane;
    static constexpr int bytes = GRAD ? At + 3 * kPlane : Tt;
};
using GradRec = Rec<true>;

// A state kept for the gradients: the C tiles of its 16-column blocks one
// after the other, as the lanes hold them (1 KB a tile).  Floats from the
// chunk's first to the lane's four of tile i of the columns from p0.
template <int NP>
__device__ __forceinline__ int64_t kept_tile(int64_t p0, int i, int lane) {
    return p0 * NP + i * 256 + lane * 4;
}

__device__ __forceinline__ int block_at(int t, int s) { return t * (t + 1) / 2 + s; }

// Tokens of batch element b.
__device__ __forceinline__ int64_t seq_len(const DeltaArgs& a, int64_t b) {
    return a.lengths ? min((int64_t)max(__builtin_amdgcn_readfirstlane(a.lengths[b]), 0), a.L) : a.L;
}

__device__ __forceinline__ float exp_f32(float x) { return fast_exp2(x * kLog2e); }

// Planes that an input of type T takes.
template <typename T> constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;

// Workgroup barrier for LDS traffic only: global loads and stores in flight
// keep running across it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What the wave's lanes wrote to LDS is there for its other lanes: LDS works
// a wave's instructions off in order, so only the compiler has to keep them.
__device__ __forceinline__ void wave_sync() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// A value that is the same in every lane, in a scalar register.  Descriptors
// have to be made of such: one in vector registers, equal in every lane or
// not, is accessed in a loop over its values (1.5 us a chunk in the scan).
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <typename T>
__device__ __forceinline__ T* scalar(T* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);   // (the builtin returns an int: its sign
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));   // must not reach the other half)
    return reinterpret_cast<T*>((uint64_t)hi << 32 | lo);
}

// A buffer over `rows` rows spaced `stride` bytes apart, of which `bytes`
// belong to it: loads past its end give zero, stores there are dropped.
// Offsets are 32-bit: 64 rows stay within 2^30 bytes (checked on the host).
constexpr int kOut = 1 << 30;   // an offset past every buffer, with room for a few rows more
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buf(const void* p, int rows, int stride, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, scalar(rows > 0 ? (rows - 1) * stride + bytes : 0), 0x00020000);
}

// Chunks of n tokens, and the tokens in chunk c of them (32-bit comparisons,
// which scalar registers allow).
struct Chunks {
    int n, last;
    __device__ __forceinline__ explicit Chunks(int64_t tokens)
        : n(scalar((int)((tokens + kC - 1) / kC))), last(scalar((int)(tokens - (tokens + kC - 1) / kC * kC + kC))) {}
    __device__ __forceinline__ int rows(int c) const { return c + 1 < n ? kC : c + 1 == n ? last : 0; }
};

// One element as loaded; widen it when it is used, not before: widening
// waits for the load.
template <typename T> __device__ __forceinline__ T buf_raw(__amdgpu_buffer_rsrc_t r, int off);
template <> __device__ __forceinline__ float buf_raw<float>(__amdgpu_buffer_rsrc_t r, int off) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}
template <> __device__ __forceinline__ uint16_t buf_raw<uint16_t>(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
}
__device__ __forceinline__ f32x4 widen(const float (&v)[4]) { return f32x4{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ f32x4 widen(const uint16_t (&v)[4]) {
    return f32x4{bf16_to_f32(v[0]), bf16_to_f32(v[1]), bf16_to_f32(v[2]), bf16_to_f32(v[3])};
}
__device__ __forceinline__ f32x4 buf_ld4(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ void buf_st(__amdgpu_buffer_rsrc_t r, int off, float v, float) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, 0, 0);
}
__device__ __forceinline__ void buf_st(__amdgpu_buffer_rsrc_t r, int off, float v, uint16_t) {
    __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v), r, off, 0, 0);
}

// Eight consecutive elements of a row as loaded, into the planes of a staged
// row (plane stride ps elements), and as an operand.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { u32x4 w; };
template <> struct Raw8<float> { f32x4 lo, hi; };

__device__ __forceinline__ void fetch8(__amdgpu_buffer_rsrc_t b, int off, Raw8<uint16_t>& r) {
    r.w = __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0);
}
__device__ __forceinline__ void fetch8(__amdgpu_buffer_rsrc_t b, int off, Raw8<float>& r) {
    r.lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
    r.hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 16, 0));
}
__device__ __forceinline__ void stage8(uint16_t* row, int ps, int n0, const Raw8<uint16_t>& r) {
    *reinterpret_cast<u32x4*>(row + n0) = r.w;
}
__device__ __forceinline__ void stage8(uint16_t* row, int ps, int n0, const Raw8<float>& r) {
    bf16x8 p[3];
    split8<3>(r.lo, r.hi, p);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x8*>(row + i * ps + n0) = p[i];
}
__device__ __forceinline__ void to_operand(const Raw8<uint16_t>& r, bf16x8 (&p)[1]) {
    p[0] = __builtin_bit_cast(bf16x8, r.w);
}
__device__ __forceinline__ void to_operand(const Raw8<float>& r, bf16x8 (&p)[3]) { split8<3>(r.lo, r.hi, p); }

__device__ __forceinline__ f32x4 sum_of(const f32x4 (&v)[2]) { return v[0] + v[1]; }
__device__ __forceinline__ f32x4 sum_of(const f32x4 (&v)[4]) { return (v[0] + v[1]) + (v[2] + v[3]); }

// B operands that waves hand to each other through LDS: NPL planes of KS
// k-steps, k in natural order, each lane's 16 bytes in its own slot.
template <int KS, int NPL>
struct Operands {
    uint16_t p[KS][NPL][64][8];
    // C tile t of the operand's rows, split.  Its lane group g holds rows
    // 16 t + 4 g ..: half g % 2 of what lane group 2 (t % 2) + g / 2 reads.
    __device__ __forceinline__ void put_tile(int t, f32x4 v, int lane) {
        uint2 w[NPL];
        split4<NPL>(v, w);
        const int at = 16 * (2 * (t & 1) + (lane >> 5)) + (lane & 15), e = 4 * ((lane >> 4) & 1);
#pragma unroll
        for (int i = 0; i < NPL; ++i) *reinterpret_cast<uint2*>(&p[t >> 1][i][at][e]) = w[i];
    }
    __device__ __forceinline__ void get(int ks, int lane, bf16x8 (&w)[NPL]) const {
#pragma unroll
        for (int i = 0; i < NPL; ++i) w[i] = ld8(p[ks][i][lane]);
    }
};

// C tiles handed through LDS as they are: a lane's four values in its slot.
struct Tiles {
    float p[4][64][4];
    __device__ __forceinline__ void put(int t, f32x4 v, int lane) { *reinterpret_cast<f32x4*>(p[t][lane]) = v; }
    __device__ __forceinline__ f32x4 get(int t, int lane) const { return *reinterpret_cast<const f32x4*>(p[t][lane]); }
};

// Byte offset in a plane of the lane's part of row block tb of T, an A
// operand: columns 32 ks + 8 g .. (kOut above the diagonal, where it is
// zero); and of row block jb of T's transpose.
__device__ __forceinline__ int row_of(int tb, int ks, int lane) {
    const int s = 2 * ks + (lane >> 5);
    return s <= tb ? block_at(tb, s) * 512 + (lane & 15) * 32 + ((lane >> 4) & 1) * 16 : kOut;
}
__device__ __forceinline__ int row_of_t(int jb, int ks, int lane) {
    const int t = 2 * ks + (lane >> 5);
    return t >= jb ? block_at(t, jb) * 512 + (lane & 15) * 32 + ((lane >> 4) & 1) * 16 : kOut;
}
__device__ __forceinline__ bf16x8 buf_op(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

}  // namespace dchunk
}  // namespace selscan
