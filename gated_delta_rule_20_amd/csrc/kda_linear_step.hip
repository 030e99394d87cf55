// kda_linear_step.hip -- one token of linear attention with a decay per head:
//   S' = exp(g) S + k v^T,   o = scale * S'^T q.
//
// Bound by moving the state once in and once out (2 x Dk x Dv x 4 bytes per
// sequence and head against 5 Dk Dv operations): every thread holds its part of
// the state in registers between one 16-byte load and one 16-byte store each.
// 512 sequences x 32 heads of 128 x 128 (2.13 GB): 391 us, 5.4 TB/s, above a copy's 4.9; 4 sequences: 4.3 us.
#include "kda_common.h"
#include "kda_linear.h"

namespace kda {

// One workgroup per (sequence, value head, COLS columns of the state).  COLS / 4
// neighbouring threads hold one row's columns (4 each), so a wave's access is
// whole 128-byte lines, and RP rows are held side by side; each thread keeps
// DK / RP rows.  o sums over rows: in the thread, across the wave, through LDS.
template <typename T, int DK, int DV, int COLS>
__global__ __launch_bounds__(256) void linear_step_kernel(const LinearStepParams p)
{
    constexpr int TPR = COLS / 4;         // threads per row
    constexpr int RP = 256 / TPR;         // rows side by side
    constexpr int NR = DK / RP;           // rows per thread
    constexpr int SPLIT = DV / COLS;
    static_assert(NR * RP == DK && NR >= 1, "rows divide evenly");
    __shared__ float s_k[DK], s_q[DK];
    __shared__ float s_o[4][COLS];

    const int t = threadIdx.x;
    const unsigned b = blockIdx.x;
    const int part = SPLIT == 1 ? 0 : (int)(b % SPLIT);
    const unsigned nh = b / SPLIT;
    const int n = (int)(nh / (unsigned)p.H), h = (int)(nh % (unsigned)p.H);
    const int c0 = part * COLS;
    int slot = n;
    bool mine = true;
    if (p.slots) {
        slot = p.slots[n];
        mine = slot >= 0 && slot < p.n_slots;
        bool seen = false;                // an earlier row of the same slot
        for (int j = t; j < n; j += 4 * 256) {             // four reads in flight
#pragma unroll
            for (int i = 0; i < 4; ++i) seen |= p.slots[min(j + 256 * i, n - 1)] == slot && j + 256 * i < n;
        }
        mine = !__syncthreads_or(seen) && mine;
    }
    if (!mine) {                          // an empty place: uniform over the workgroup
        if (t < COLS) ((T *)p.o)[(size_t)nh * DV + c0 + t] = from_f<T>(0.f);
        return;
    }
    const int r0 = t / TPR, c = c0 + 4 * (t % TPR);
    const size_t base = ((size_t)slot * p.H + h) * (size_t)(DK * DV) + (size_t)r0 * DV + c;
    f32x4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p.state + base + (size_t)i * RP * DV));
    const size_t kv = ((size_t)n * (p.H / p.group) + h / p.group) * DK;
    if (t < DK) s_k[t] = to_f<T>(((const T *)p.k)[kv + t]);
    if (t >= 256 - DK) s_q[t - (256 - DK)] = to_f<T>(((const T *)p.q)[kv + t - (256 - DK)]);
    const quad_t<T> vq = *reinterpret_cast<const quad_t<T> *>((const T *)p.v + (size_t)nh * DV + c);
    const f32x4 v = quad_to_f<T>(vq);
    const float e = __builtin_amdgcn_exp2f(log2_decay(p.g[p.g_per_head ? h : (int)nh]));
    __syncthreads();
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const float k = s_k[r0 + i * RP], q = s_q[r0 + i * RP];
        s[i] = s[i] * e + v * k;
        o += s[i] * q;
        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4 *>(p.new_state + base + (size_t)i * RP * DV));
    }
#pragma unroll
    for (int d = TPR; d < 64; d *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], d);
    if ((t & 63) < TPR) *reinterpret_cast<f32x4 *>(&s_o[t >> 6][4 * (t % TPR)]) = o;
    __syncthreads();
    if (t < COLS)
        ((T *)p.o)[(size_t)nh * DV + c0 + t] =
            from_f<T>(p.scale * ((s_o[0][t] + s_o[1][t]) + (s_o[2][t] + s_o[3][t])));
}

template <typename T, int DK, int DV> static hipError_t launch_step_t(const LinearStepParams &p, hipStream_t stream)
{
    const unsigned pairs = (unsigned)((size_t)p.N * p.H);
    // Fewer (sequence, head) pairs than compute units: columns split, four times the workgroups.
    if (pairs < 256)
        hipLaunchKernelGGL((linear_step_kernel<T, DK, DV, 32>), dim3(pairs * (DV / 32)), dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((linear_step_kernel<T, DK, DV, DV>), dim3(pairs), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_linear_step(int dtype_bf16, int Dk, int Dv, const LinearStepParams &p, hipStream_t stream)
{
#define KDA_STEP_CASE(TT, DKV, DVV) \
    if (Dk == DKV && Dv == DVV) return launch_step_t<TT, DKV, DVV>(p, stream);
    if (dtype_bf16) {
        KDA_STEP_CASE(bf16, 64, 64)
        KDA_STEP_CASE(bf16, 64, 128)
        KDA_STEP_CASE(bf16, 128, 64)
        KDA_STEP_CASE(bf16, 128, 128)
    } else {
        KDA_STEP_CASE(float, 64, 64)
        KDA_STEP_CASE(float, 64, 128)
        KDA_STEP_CASE(float, 128, 64)
        KDA_STEP_CASE(float, 128, 128)
    }
#undef KDA_STEP_CASE
    return hipErrorInvalidValue;
}

}  // namespace kda
