// Compares the element helpers' scale and reciprocal with CUDA's correctly rounded division
// and reciprocal, for every finite maximum and every scale that one gives.  Prints the
// number of differences of each.
#include <cstdio>

#include "rlq_elem.cuh"

namespace {

// Bit patterns first .. last, a grid-stride loop; wrong[0]: scales, wrong[1]: reciprocals.
__global__ void compare(unsigned long long first, unsigned long long last, unsigned long long *wrong)
{
    unsigned long long scales = 0, rcps = 0;
    const unsigned long long step = (unsigned long long)gridDim.x * blockDim.x;
    for (unsigned long long b = first + (unsigned long long)blockIdx.x * blockDim.x + threadIdx.x; b <= last; b += step) {
        const float a = __uint_as_float((unsigned)b);
        const float q = __fdiv_rn(a, 448.0f);
        const float want = a == 0.0f ? 1.0f : q == 0.0f ? __uint_as_float(1u) : q;
        scales += __float_as_uint(rlq::group_scale(a)) != __float_as_uint(want);
        // as a scale: those that a finite maximum gives
        if (a > 0.0f && a <= __fdiv_rn(__uint_as_float(0x7F7FFFFFu), 448.0f)) {
            const float d = a * rlq::scale_pre(a);
            rcps += __float_as_uint(rlq::scale_rcp(a)) != __float_as_uint(__frcp_rn(d));
        }
    }
    if (scales)
        atomicAdd(wrong, scales);
    if (rcps)
        atomicAdd(wrong + 1, rcps);
}

}  // namespace

int main()
{
    unsigned long long *wrong, got[2] = {1, 1};
    if (cudaMalloc(&wrong, sizeof got) != cudaSuccess || cudaMemset(wrong, 0, sizeof got) != cudaSuccess)
        return 2;
    compare<<<1216, 256>>>(0ull, 0x7F7FFFFFull, wrong);
    if (cudaGetLastError() != cudaSuccess || cudaMemcpy(got, wrong, sizeof got, cudaMemcpyDeviceToHost) != cudaSuccess)
        return 3;
    std::printf("%llu %llu\n", got[0], got[1]);
    return cudaFree(wrong) == cudaSuccess ? 0 : 4;
}
