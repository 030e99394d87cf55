// kda_scan.hip -- the gated scan  h_t = a_t h_{t-1} + m_t x_t  per channel:
// whole sequences, their gradients, one token.
#include "kda_block_dev.h"

namespace kda {

// The log-decay a token's g stands for; with logits (eq. (5)) its gate too.
struct Gate {
    float eA, g_min;
    bool on;
    __device__ __forceinline__ float log_decay(float g) const { return on ? g_min * sigmoid2(eA * g).s : g; }
    // d log_decay / d g
    __device__ __forceinline__ float slope(float g) const
    {
        if (!on) return 1.f;
        const Sigmoid s = sigmoid2(eA * g);
        return g_min * s.s * s.r * eA;
    }
};

__device__ __forceinline__ Gate gate_of(const float *A_log, float g_min, int c)
{
    Gate g;
    g.on = A_log != nullptr;
    g.eA = g.on ? __expf(A_log[c]) : 1.f;
    g.g_min = g_min;
    return g;
}

// Rows [lo, hi) of sequence s.
__device__ __forceinline__ void sequence_of(const ScanParams &p, int s, int *lo, int *hi)
{
    if (!p.cu) {
        *lo = s * p.T;
        *hi = *lo + p.T;
        return;
    }
    *lo = min(max(p.cu[s], 0), p.rows);
    *hi = min(max(p.cu[s + 1], *lo), p.rows);
}

template <typename T, typename G> __global__ __launch_bounds__(64) void scan_fwd_kernel(const ScanParams p)
{
    const int blocks = (p.C + 63) / 64;
    const int s = blockIdx.x / blocks, c = (blockIdx.x % blocks) * 64 + threadIdx.x;
    if (c >= p.C) return;
    int lo, hi;
    sequence_of(p, s, &lo, &hi);
    const Gate gate = gate_of(p.A_log, p.g_min, c);
    float h = p.h0 ? p.h0[(size_t)s * p.C + c] : 0.f;
    for (int t = lo; t < hi; ++t) {
        const float w = decay_code(gate.log_decay(to_f<G>(((const G *)p.g.p)[t * p.g.stride + c])));
        float x = to_f<T>(((const T *)p.x.p)[t * p.x.stride + c]);
        if (p.complement) x *= decay_rest(w);
        h = decay_apply(w, h, x);
        ((T *)p.h)[(size_t)t * p.C + c] = from_f<T>(h);
    }
    if (p.hT) p.hT[(size_t)s * p.C + c] = h;
}

template <typename T> __device__ __forceinline__ float load_one(const Rows &m, size_t r, int C, int c)
{
    if (m.scales) return (float)((const int8_t *)m.p)[r * m.stride + c] * m.scales[r * act_groups(C) + c / ACT_GROUP];
    return to_f<T>(((const T *)m.p)[r * m.stride + c]);
}

template <typename T, typename G> __global__ __launch_bounds__(64) void scan_bwd_kernel(const ScanParams p)
{
    const int blocks = (p.C + 63) / 64;
    const int s = blockIdx.x / blocks, c = (blockIdx.x % blocks) * 64 + threadIdx.x;
    if (c >= p.C) return;
    int lo, hi;
    sequence_of(p, s, &lo, &hi);
    const Gate gate = gate_of(p.A_log, p.g_min, c);
    float e = p.dhT ? p.dhT[(size_t)s * p.C + c] : 0.f, dA = 0.f;
    for (int t = hi - 1; t >= lo; --t) {
        const float z = to_f<G>(((const G *)p.g.p)[t * p.g.stride + c]);
        const float w = decay_code(gate.log_decay(z));
        const float D = to_f<T>(((const T *)p.d_h)[(size_t)t * p.C + c]) + e;
        e = decay_times(w, D);
        ((T *)p.dx)[t * p.dx_stride + c] = from_f<T>(p.complement ? D * decay_rest(w) : D);
        if (p.dg) {
            float prev = t > lo ? load_one<T>(p.hs, t - 1, p.C, c) : p.h0 ? p.h0[(size_t)s * p.C + c] : 0.f;
            if (p.complement) prev -= load_one<T>(p.x, t, p.C, c);
            const float dz = e * prev * gate.slope(z);
            ((G *)p.dg)[t * p.dg_stride + c] = from_f<G>(dz);
            dA += dz * z;
        }
    }
    if (p.dh0) p.dh0[(size_t)s * p.C + c] = e;
    if (p.dA_part) p.dA_part[(size_t)s * p.C + c] = dA;
}

__global__ __launch_bounds__(64) void scan_sum_kernel(const float *part, int parts, int C, float *out)
{
    const int c = blockIdx.x * 64 + threadIdx.x;
    if (c >= C) return;
    double sum = 0.0;
    for (int i = 0; i < parts; ++i) sum += part[(size_t)i * C + c];
    out[c] = (float)sum;
}

// One token a sequence: 8 channels a lane.  Slots as for kda_linear_recurrent_step.
template <typename T, typename G> __global__ __launch_bounds__(256) void scan_step_kernel(const ScanStepParams p)
{
    const int blocks = (p.C + 2047) / 2048;
    const int n = blockIdx.x / blocks, c = (blockIdx.x % blocks) * 2048 + threadIdx.x * LANE_CH;
    const int cnt = max(0, min(LANE_CH, p.C - c));
    int slot = n;
    bool mine = true;
    if (p.slots) {
        slot = p.slots[n];
        mine = slot >= 0 && slot < p.n_slots;
        bool seen = false;
        for (int j = threadIdx.x; j < n; j += 256) seen |= p.slots[j] == slot;
        mine = !__syncthreads_or(seen) && mine;
    }
    if (cnt == 0) return;
    float h[8];
    if (mine) {
        Raw8<T> x;
        Raw8<G> g;
        float A[8];
        x.load((const T *)p.x.p + n * p.x.stride + c, cnt);
        g.load((const G *)p.g.p + n * p.g.stride + c, cnt);
        load_f8(p.state + (size_t)slot * p.C + c, cnt, h);
        if (p.A_log) load_f8(p.A_log + c, cnt, A);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Gate gate = {p.A_log ? __expf(A[i]) : 1.f, p.g_min, p.A_log != nullptr};
            const float w = decay_code(gate.log_decay(g[i]));
            h[i] = decay_apply(w, h[i], p.complement ? x[i] * decay_rest(w) : x[i]);
        }
        Raw8<float>::store(p.new_state + (size_t)slot * p.C + c, cnt, h);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = 0.f;
    }
    Raw8<T>::store((T *)p.h + (size_t)n * p.C + c, cnt, h);
}

template <typename T, typename G> static hipError_t launch_fwd_t(const ScanParams &p, hipStream_t stream)
{
    hipLaunchKernelGGL((scan_fwd_kernel<T, G>), dim3((unsigned)p.N * ((p.C + 63) / 64)), dim3(64), 0, stream, p);
    if (p.h8.codes && p.rows > 0) {
        const Rows h = {p.h, nullptr, p.C};
        return launch_act_pack(sizeof(T) == 2, h, p.rows, p.C, p.h8, stream, p.cu, p.cu ? p.cu + p.N : nullptr);
    }
    return hipGetLastError();
}

template <typename T, typename G> static hipError_t launch_bwd_t(const ScanParams &p, hipStream_t stream)
{
    hipLaunchKernelGGL((scan_bwd_kernel<T, G>), dim3((unsigned)p.N * ((p.C + 63) / 64)), dim3(64), 0, stream, p);
    if (p.dA) hipLaunchKernelGGL(scan_sum_kernel, dim3((p.C + 63) / 64), dim3(64), 0, stream, p.dA_part, p.N, p.C, p.dA);
    return hipGetLastError();
}

template <typename T, typename G> static hipError_t launch_step_t(const ScanStepParams &p, hipStream_t stream)
{
    hipLaunchKernelGGL((scan_step_kernel<T, G>), dim3((unsigned)p.N * ((p.C + 2047) / 2048)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

#define KDA_SCAN_CASE(fn)                                                                       \
    return !is_bf16 ? fn<float, float>(p, stream) : g_bf16 ? fn<bf16, bf16>(p, stream) : fn<bf16, float>(p, stream)

hipError_t launch_scan_fwd(int is_bf16, int g_bf16, const ScanParams &p, hipStream_t stream) { KDA_SCAN_CASE(launch_fwd_t); }
hipError_t launch_scan_bwd(int is_bf16, int g_bf16, const ScanParams &p, hipStream_t stream) { KDA_SCAN_CASE(launch_bwd_t); }
hipError_t launch_scan_step(int is_bf16, int g_bf16, const ScanStepParams &p, hipStream_t stream) { KDA_SCAN_CASE(launch_step_t); }

#undef KDA_SCAN_CASE

}  // namespace kda
