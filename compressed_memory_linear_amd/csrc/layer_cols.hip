// layer_cols.hip -- column sums of workgroups' partial sums.
#include "layer_device.h"
#include "layer_launch.h"

namespace layer {
namespace {

// One row of the sum, 32 columns and 32 rows of threads to a workgroup: each thread adds every 32nd
// group in order, 16 loads at a time, then a tree over the rows of threads.
__global__ __launch_bounds__(1024) void layer_cols_kernel(ColSums p) {
    __shared__ float s[32][32];
    const int row = blockIdx.y;
    float* out = row < p.M ? p.mat : row == p.M ? p.e0 : p.e1;
    if (!out) return;
    const int64_t step = row < p.M ? p.M : 1;
    const int l = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + l;
    const int64_t pitch = static_cast<int64_t>(p.rows) * p.D;
    const float* part = p.part + static_cast<int64_t>(row) * p.D + c;
    float a = 0.0f;
    for (int g0 = r; g0 < p.groups; g0 += 32 * 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = c < p.D && g0 + 32 * i < p.groups ? part[(g0 + 32 * i) * pitch] : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a += v[i];
    }
    s[r][l] = a;
#pragma unroll
    for (int n = 16; n > 0; n /= 2) {
        __syncthreads();
        if (r < n) s[r][l] += s[r + n][l];
    }
    if (r == 0 && c < p.D) out[c * step + (row < p.M ? row : 0)] = s[0][l];
}

}  // namespace

void launch_col_sums(const ColSums& p, hipStream_t st) {
    hipLaunchKernelGGL(layer_cols_kernel, dim3((p.D + 31) / 32, p.rows), dim3(1024), 0, st, p);
}

}  // namespace layer
