// kda_block_norm.hip -- what stands between two blocks of a model:
//   u = w_post y / rms(y),  x' = x + s Sigmoid(gate) u,  n = w_pre x' / rms(x'),
// and its gradients.
#include "kda_block_dev.h"

namespace kda {

// Sums of K values over the NW waves that hold a row, on every lane.  The waves' sums pass through LDS; two
// buffers in turn, so that one barrier a sum is enough.
template <int NW, int K> struct RowSum {
    float (*lds)[NW][K];
    int turn;
    __device__ __forceinline__ void operator()(float *v)
    {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
        if constexpr (NW > 1) {
            const int wave = threadIdx.x / 64;
            if (lane_id() == 0)
#pragma unroll
                for (int k = 0; k < K; ++k) lds[turn][wave][k] = v[k];
            lds_barrier();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                v[k] = lds[turn][0][k];
#pragma unroll
                for (int w = 1; w < NW; ++w) v[k] += lds[turn][w][k];
            }
            turn ^= 1;
        }
    }
};

constexpr int norm_threads(int nw) { return nw == 1 ? 256 : 64 * nw; }

template <typename T, typename X, int NW, int NCH>
__global__ __launch_bounds__(norm_threads(NW)) void norm_fwd_kernel(const NormParams p)
{
    constexpr int NT = 64 * NW;                            // threads of a row
    constexpr int ROWS = norm_threads(NW) / NT;            // rows side by side
    __shared__ float s_sum[2][NW][1];
    RowSum<NW, 1> sum = {s_sum, 0};
    const int t = threadIdx.x % NT;
    int cnt[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) cnt[j] = max(0, min(LANE_CH, p.D - (j * NT + t) * LANE_CH));
    for (int row = blockIdx.x * ROWS + threadIdx.x / NT; row < p.R; row += gridDim.x * ROWS) {
        const size_t r = row;
        float u[NCH][8], x[NCH][8];
        float ss[1] = {0.f};
        if (p.y.p) {
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = (j * NT + t) * LANE_CH;
                load_row8<T>(p.y, r, p.D, c, cnt[j], u[j]);
                if (p.y8.codes) store_codes<LANE_CH>(p.y8, r, p.D, c, cnt[j], u[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] += u[j][i] * u[j][i];
            }
            float rs = 1.f;
            if (p.post) {
                sum(ss);
                rs = rstd_of(ss[0] / (float)p.D + p.eps);
            }
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = (j * NT + t) * LANE_CH;
                float w[8];
                if (p.post) {
                    load_f8(p.post + c, cnt[j], w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[j][i] = w[i] * (u[j][i] * rs);
                }
                if (p.gate.p) {
                    load_row8<T>(p.gate, r, p.D, c, cnt[j], w);
                    if (p.gate8.codes) store_codes<LANE_CH>(p.gate8, r, p.D, c, cnt[j], w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[j][i] *= sigmoid2(w[i]).s;
                }
                if (p.res) {
                    load_f8(p.res + c, cnt[j], w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[j][i] *= w[i];
                }
            }
        }
        ss[0] = 0.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = (j * NT + t) * LANE_CH;
            load_row8<X>(p.x, r, p.D, c, cnt[j], x[j]);
            if (p.y.p) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = to_f<X>(from_f<X>(x[j][i] + p.scale * u[j][i]));
                if (cnt[j] > 0) Raw8<X>::store((X *)p.x_out + r * p.D + c, cnt[j], x[j]);
            }
            if (p.x8.codes) store_codes<LANE_CH>(p.x8, r, p.D, c, cnt[j], x[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] += x[j][i] * x[j][i];
        }
        if (p.pre) {
            sum(ss);
            const float rs = rstd_of(ss[0] / (float)p.D + p.eps);
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = (j * NT + t) * LANE_CH;
                float w[8];
                load_f8(p.pre + c, cnt[j], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] *= x[j][i] * rs;
                if (cnt[j] > 0) Raw8<T>::store((T *)p.n + r * p.D + c, cnt[j], w);
            }
        }
    }
}

template <typename T, typename X, int NW, int NCH>
__global__ __launch_bounds__(norm_threads(NW)) void norm_bwd_kernel(const NormParams p)
{
    constexpr int NT = 64 * NW;
    constexpr int ROWS = norm_threads(NW) / NT;
    __shared__ float s_sum[2][NW][3];
    __shared__ float s_one[2][NW][1];
    RowSum<NW, 3> sum3 = {s_sum, 0};
    RowSum<NW, 1> sum1 = {s_one, 0};
    const int t = threadIdx.x % NT;
    const int part = blockIdx.x * ROWS + threadIdx.x / NT;
    int cnt[NCH];
    float a_post[NCH][8] = {}, a_res[NCH][8] = {}, a_pre[NCH][8] = {};
#pragma unroll
    for (int j = 0; j < NCH; ++j) cnt[j] = max(0, min(LANE_CH, p.D - (j * NT + t) * LANE_CH));
    const float inv_d = 1.f / (float)p.D;
    for (int row = part < p.parts ? part : p.R; row < p.R; row += p.parts) {
        const size_t r = row;
        float x[NCH][8], dn[NCH][8], y[NCH][8];
        float s3[3] = {0.f, 0.f, 0.f};                     // y^2, x^2, w_pre dn x
        const bool pre = p.pre && p.d_n;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = (j * NT + t) * LANE_CH;
            if (p.y.p) {
                load_row8<T>(p.y, r, p.D, c, cnt[j], y[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s3[0] += y[j][i] * y[j][i];
            }
            if (pre) {
                const Rows d = {p.d_n, nullptr, p.D};
                float w[8];
                load_row8<X>(p.x, r, p.D, c, cnt[j], x[j]);
                load_row8<T>(d, r, p.D, c, cnt[j], dn[j]);
                load_f8(p.pre + c, cnt[j], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s3[1] += x[j][i] * x[j][i];
                    s3[2] += w[i] * dn[j][i] * x[j][i];
                }
            }
        }
        sum3(s3);
        const float ry = p.post ? rstd_of(s3[0] * inv_d + p.eps) : 1.f;
        const float rx = rstd_of(s3[1] * inv_d + p.eps);
        const float mx = s3[2] * rx * inv_d;               // mean of w_pre dn x^
        float s1[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = (j * NT + t) * LANE_CH;
            float G[8], w[8];
            if (p.d_x) {
                const Rows d = {p.d_x, nullptr, p.D};
                load_row8<X>(d, r, p.D, c, cnt[j], G);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) G[i] = 0.f;
            }
            if (pre) {
                load_f8(p.pre + c, cnt[j], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = x[j][i] * rx;
                    a_pre[j][i] += dn[j][i] * xh;
                    G[i] += rx * (w[i] * dn[j][i] - xh * mx);
                }
            }
            if (cnt[j] > 0) Raw8<X>::store((X *)p.dx + r * p.D + c, cnt[j], G);
            if (!p.y.p) continue;
            float u[8], res[8], gt[8];
            if (p.post) load_f8(p.post + c, cnt[j], w);
            if (p.res) load_f8(p.res + c, cnt[j], res);
            if (p.gate.p) load_row8<T>(p.gate, r, p.D, c, cnt[j], gt);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[j][i] *= ry;
                u[i] = p.post ? w[i] * y[j][i] : y[j][i];
                const Sigmoid s = p.gate.p ? sigmoid2(gt[i]) : Sigmoid{1.f, 0.f};
                float dr = G[i] * p.scale;
                a_res[j][i] += dr * (s.s * u[i]);
                if (p.res) dr *= res[i];
                gt[i] = dr * u[i] * (s.s * s.r);
                float du = dr * s.s;
                if (p.post) {
                    a_post[j][i] += du * y[j][i];
                    du *= w[i];
                    s1[0] += du * y[j][i];
                }
                dn[j][i] = du;
            }
            if (p.gate.p && cnt[j] > 0) Raw8<T>::store((T *)p.dgate + r * p.dgate_stride + c, cnt[j], gt);
        }
        if (!p.y.p) continue;
        float my = 0.f;
        if (p.post) {
            sum1(s1);
            my = s1[0] * inv_d;
        }
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = (j * NT + t) * LANE_CH;
            if (p.post)
#pragma unroll
                for (int i = 0; i < 8; ++i) dn[j][i] = ry * (dn[j][i] - y[j][i] * my);
            if (cnt[j] > 0) Raw8<T>::store((T *)p.dy + r * p.dy_stride + c, cnt[j], dn[j]);
        }
    }
    if (part >= p.parts) return;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        const int c = (j * NT + t) * LANE_CH;
        if (cnt[j] == 0) continue;
        float *at = p.part + (size_t)part * p.D + c;
        const size_t step = (size_t)p.parts * p.D;
        if (p.dpost) Raw8<float>::store(at, cnt[j], a_post[j]);
        if (p.dres) Raw8<float>::store(at + step, cnt[j], a_res[j]);
        if (p.dpre) Raw8<float>::store(at + 2 * step, cnt[j], a_pre[j]);
    }
}

// The weights' gradients from the workgroups' sums, in their order.
__global__ __launch_bounds__(256) void norm_sum_kernel(const NormParams p)
{
    __shared__ double s_part[4][64];
    float *out = blockIdx.y == 0 ? p.dpost : blockIdx.y == 1 ? p.dres : p.dpre;
    if (!out) return;
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), slice = threadIdx.x / 64;
    const float *at = p.part + (size_t)blockIdx.y * p.parts * p.D + c;
    double sum = 0.0;
    if (c < p.D)
        for (int i = slice; i < p.parts; i += 4) sum += at[(size_t)i * p.D];
    s_part[slice][threadIdx.x & 63] = sum;
    __syncthreads();
    if (slice == 0 && c < p.D) {
        const int l = threadIdx.x;
        out[c] = (float)((s_part[0][l] + s_part[1][l]) + (s_part[2][l] + s_part[3][l]));
    }
}

// Threads for a row: 8 channels a lane, up to 16 waves, then twice that.
template <template <typename, typename, int, int> class K, typename T, typename X>
static hipError_t launch_by_width(const NormParams &p, hipStream_t stream)
{
    if (p.D <= 512) return K<T, X, 1, 1>::launch(p, stream);
    if (p.D <= 1024) return K<T, X, 2, 1>::launch(p, stream);
    if (p.D <= 2048) return K<T, X, 4, 1>::launch(p, stream);
    if (p.D <= 4096) return K<T, X, 8, 1>::launch(p, stream);
    if (p.D <= 8192) return K<T, X, 16, 1>::launch(p, stream);
    return K<T, X, 16, 2>::launch(p, stream);
}

template <typename T, typename X, int NW, int NCH> struct Fwd {
    static hipError_t launch(const NormParams &p, hipStream_t stream)
    {
        constexpr int rows = norm_threads(NW) / (64 * NW);
        const int grid = (p.R + rows - 1) / rows;
        hipLaunchKernelGGL((norm_fwd_kernel<T, X, NW, NCH>), dim3(grid < 2048 ? grid : 2048), dim3(norm_threads(NW)), 0, stream, p);
        return hipGetLastError();
    }
};

template <typename T, typename X, int NW, int NCH> struct Bwd {
    static hipError_t launch(const NormParams &p, hipStream_t stream)
    {
        constexpr int rows = norm_threads(NW) / (64 * NW);
        if (p.R > 0)
            hipLaunchKernelGGL((norm_bwd_kernel<T, X, NW, NCH>), dim3((p.parts + rows - 1) / rows), dim3(norm_threads(NW)), 0, stream, p);
        if (p.dpost || p.dres || p.dpre)
            hipLaunchKernelGGL(norm_sum_kernel, dim3((p.D + 63) / 64, 3), dim3(256), 0, stream, p);
        return hipGetLastError();
    }
};

hipError_t launch_norm_fwd(int is_bf16, int x_bf16, const NormParams &p, hipStream_t stream)
{
    if (!is_bf16) return launch_by_width<Fwd, float, float>(p, stream);
    return x_bf16 ? launch_by_width<Fwd, bf16, bf16>(p, stream) : launch_by_width<Fwd, bf16, float>(p, stream);
}

hipError_t launch_norm_bwd(int is_bf16, int x_bf16, const NormParams &p, hipStream_t stream)
{
    if (!is_bf16) return launch_by_width<Bwd, float, float>(p, stream);
    return x_bf16 ? launch_by_width<Bwd, bf16, bf16>(p, stream) : launch_by_width<Bwd, bf16, float>(p, stream);
}

}  // namespace kda
