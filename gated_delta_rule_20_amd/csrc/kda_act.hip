// kda_act.hip -- activations in 8 bits: packing and unpacking rows.
#include "kda_block_dev.h"

namespace kda {

// A lane packs 8 channels (one 16-byte load of bf16), 16 lanes a group, so that its largest value is four steps among the lanes of a
// row of the register file; a workgroup takes 16 groups of consecutive rows' groups.  Bound by memory: 8192 x 4096 in bf16 packs in
// 21 us (102 MB, 4.9 TB/s) and unpacks in 17.3 (5.9 TB/s, the codes partly from a cache).
template <typename T> __global__ __launch_bounds__(256) void act_pack_kernel(Rows x, long long groups, int D, PackedOut out)
{
    const int per = act_groups(D);
    const long long at = (long long)blockIdx.x * 16 + threadIdx.x / 16;
    const bool in = at < groups;
    const size_t r = in ? (size_t)(at / per) : 0;
    const int c = in ? (int)(at % per) * ACT_GROUP + (threadIdx.x & 15) * LANE_CH : 0;
    const int n = in ? max(0, min(LANE_CH, D - c)) : 0;
    float v[8];
    Raw8<T> raw;
    raw.load((const T *)x.p + r * x.stride + c, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = raw[i];
    store_codes<LANE_CH>(out, r, D, c, n, v);
}

template <typename T> __global__ __launch_bounds__(256) void act_unpack_kernel(Rows x, long long groups, int D, T *out)
{
    const int per = act_groups(D);
    const long long at = (long long)blockIdx.x * 16 + threadIdx.x / 16;
    if (at >= groups) return;
    const size_t r = (size_t)(at / per);
    const int c = (int)(at % per) * ACT_GROUP + (threadIdx.x & 15) * LANE_CH;
    const int n = max(0, min(LANE_CH, D - c));
    float v[8];
    load_codes((const int8_t *)x.p + r * x.stride, x.scales + r * per, c, n, v);
    if (n > 0) Raw8<T>::store(out + r * D + c, n, v);
}

hipError_t launch_act_pack(int is_bf16, const Rows &x, long long rows, int D, const PackedOut &out, hipStream_t stream)
{
    const long long groups = rows * ((D + ACT_GROUP - 1) / ACT_GROUP);
    const dim3 grid((unsigned)((groups + 15) / 16));
    if (is_bf16)
        hipLaunchKernelGGL((act_pack_kernel<bf16>), grid, dim3(256), 0, stream, x, groups, D, out);
    else
        hipLaunchKernelGGL((act_pack_kernel<float>), grid, dim3(256), 0, stream, x, groups, D, out);
    return hipGetLastError();
}

hipError_t launch_act_unpack(int is_bf16, const Rows &x, long long rows, int D, void *out, hipStream_t stream)
{
    const long long groups = rows * ((D + ACT_GROUP - 1) / ACT_GROUP);
    const dim3 grid((unsigned)((groups + 15) / 16));
    if (is_bf16)
        hipLaunchKernelGGL((act_unpack_kernel<bf16>), grid, dim3(256), 0, stream, x, groups, D, (bf16 *)out);
    else
        hipLaunchKernelGGL((act_unpack_kernel<float>), grid, dim3(256), 0, stream, x, groups, D, (float *)out);
    return hipGetLastError();
}

}  // namespace kda
