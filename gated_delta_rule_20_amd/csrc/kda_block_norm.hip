// kda_block_norm.hip -- what stands between two blocks of a model:
//   u = w_post y / rms(y),  x' = x + s Sigmoid(gate) u,  n = w_pre x' / rms(x'),
// and its gradients.
#include "kda_block_dev.h"

namespace kda {

// The sum of a value over the NW waves that hold a row, on every lane.  The waves' sums pass through LDS, where each
// 16 lanes read one a lane and add them up among themselves; two buffers in turn, so that one barrier a sum is enough.
template <int NW> struct RowSum {
    float (*lds)[NW];
    int turn;
    __device__ __forceinline__ float operator()(float v)
    {
        v = wave_sum(v);
        if constexpr (NW > 1) {
            const int wave = threadIdx.x / 64 % NW;        // of the row
            if (lane_id() == 0) lds[turn][wave] = v;
            lds_barrier();
            const int w = threadIdx.x % 16;
            float x = lds[turn][w % NW];
            x = w < NW ? x : 0.f;
            x = dpp_add<0xB1, 0xF>(x);                     // quad_perm [1, 0, 3, 2]
            x = dpp_add<0x4E, 0xF>(x);                     // quad_perm [2, 3, 0, 1]
            x = dpp_add<0x141, 0xF>(x);                    // row_half_mirror
            v = dpp_add<0x140, 0xF>(x);                    // row_mirror
            turn ^= 1;
        }
        return v;
    }
};

// Six such sums at once: lanes trade values while they add (8, 4, 2 of them a lane), so that a wave needs 30 instructions
// instead of 42 and the waves' sums 14 instead of 30; uniform results.
__device__ __forceinline__ float rows_add(float v)                                    // over the four rows of 16 lanes
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    auto a = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t c = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]));
    a = __builtin_amdgcn_permlane32_swap(c, c, false, false);
    return __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
}
template <int NW> struct RowSum6 {
    float (*lds)[NW][8];
    int turn;
    __device__ __forceinline__ void operator()(float *v)
    {
        const int lane = lane_id();
        const bool odd = lane & 1, high = lane & 2;
        float a[4], b[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {                       // value k or k + 4
            const float other = k < 2 ? v[k + 4] : 0.f;
            a[k] = (odd ? other : v[k]) + dpp_move<0xB1>(odd ? v[k] : other);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            b[k] = (high ? a[k + 2] : a[k]) + dpp_move<0x4E>(high ? a[k] : a[k + 2]);
            b[k] = dpp_add<0x128, 0xF>(b[k]);               // row_ror:8
            b[k] = dpp_add<0x124, 0xF>(b[k]);               // row_ror:4
            b[k] = rows_add(b[k]);
        }
        // lane l now has values 4 (l & 1) + (l & 2) and the next one
        if constexpr (NW == 1) {
#pragma unroll
            for (int k = 0; k < 6; ++k) v[k] = read_lane(b[k % 2], k / 4 + (k & 2));
        } else {
            const int wave = threadIdx.x / 64 % NW;
            if (lane < 4) {
                lds[turn][wave][4 * (lane & 1) + (lane & 2)] = b[0];
                lds[turn][wave][4 * (lane & 1) + (lane & 2) + 1] = b[1];
            }
            lds_barrier();
            float x = lds[turn][lane / 8 % NW][lane % 8];
            if (NW == 16) x += lds[turn][(lane / 8 + 8) % NW][lane % 8];
            if (NW < 8) x = lane / 8 < NW ? x : 0.f;
            x = rows_add(dpp_add<0x128, 0xF>(x));
#pragma unroll
            for (int k = 0; k < 6; ++k) v[k] = read_lane(x, k);
            turn ^= 1;
        }
    }
    template <int CTRL> __device__ static __forceinline__ float dpp_move(float v)
    {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
    }
    __device__ static __forceinline__ float read_lane(float v, int l)
    {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
    }
};

template <int V, typename A, typename B> struct Pick { typedef A type; };
template <typename A, typename B> struct Pick<8, A, B> { typedef B type; };

// A uniform address and a lane's 32-bit offset.
template <typename T> __device__ __forceinline__ T *at_byte(T *p, unsigned bytes)
{
    return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(p) + bytes);
}

// V (4 or 8) channels of a row as they are stored: elements, or codes with their scale.
template <typename T, int V> struct HeldV {
    static constexpr int WORDS = V * sizeof(T) / 4;
    typedef typename Pick<V, Raw4<T>, Raw8<T>>::type Raw;
    uint32_t v[WORDS];
    // Channels [c, c + n), r uniform; or all V from `from` on, before c, with c's scale.
    __device__ __forceinline__ void load(const Rows &m, size_t r, int D, unsigned c, unsigned from, int n)
    {
        if (m.scales) {
            const int8_t *at = (const int8_t *)m.p + r * m.stride + from;
            if (n == V) {
                typedef uint32_t codes_any __attribute__((ext_vector_type(V / 4), aligned(1)));
                const codes_any q = *reinterpret_cast<const codes_any *>(at);
#pragma unroll
                for (int k = 0; k < V / 4; ++k) v[k] = q[k];
            } else {
                v[0] = v[V / 4 - 1] = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < n) v[i / 4] |= (uint32_t)(uint8_t)at[i] << (8 * (i % 4));
            }
            v[V / 4] = n > 0 ? __builtin_bit_cast(uint32_t, *at_byte(m.scales + r * act_groups(D), c / ACT_GROUP * 4)) : 0;
            return;
        }
        Raw raw;
        raw.load(at_byte((const T *)m.p + r * m.stride, from * sizeof(T)), n);
        __builtin_memcpy(v, &raw, sizeof(raw));
    }
    // Takes the first e of four channels off, zeros behind the others.
    __device__ __forceinline__ void drop(bool packed, int e)
    {
        static_assert(V == 4, "codes of one word");
        if (packed) {
            v[0] >>= 8 * e;
            return;
        }
        if (sizeof(T) == 2) {
            const uint64_t q = ((uint64_t)v[1] << 32 | v[0]) >> 16 * e;
            v[0] = (uint32_t)q;
            v[1] = (uint32_t)(q >> 32);
            return;
        }
#pragma unroll
        for (int step = 1; step < WORDS; step *= 2)
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const uint32_t other = i + step < WORDS ? v[i + step] : 0;
                v[i] = e & step ? other : v[i];
            }
    }
    // channels [4 k, 4 k + 4)
    __device__ __forceinline__ void get(bool packed, int k, float *x) const
    {
        if (packed) {
            const float s = __builtin_bit_cast(float, v[V / 4]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(v[k] >> (8 * i)) * s;
            return;
        }
        Raw raw;
        __builtin_memcpy(&raw, v, sizeof(raw));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = raw[4 * k + i];
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) v[i] = 0;
    }
    __device__ __forceinline__ void hold()                 // what is made from these words is not kept
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(v[i]));
    }
};

// A weight's channels of a lane, `otherwise` where there is no weight.
__device__ __forceinline__ void load_weight(const float *w, int c, int n, float otherwise, float *x)
{
    if (w) {
        load_f8(w + c, n, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = otherwise;
}

// Forward.  Bound by memory, 10 bytes an element in bf16: 8192 x 4096 62 to 66 us (336 MB, 5.1 TB/s or more).  NW waves hold a row, 8 NCH channels
// a lane (16-byte loads of bf16); a workgroup of ROWS such rows side by side goes through its rows with the weights in registers and
// the next rows' values on their way.

template <typename T, typename X, int NW, int ROWS, int NCH>
__global__ __launch_bounds__(64 * NW * ROWS, 4) void norm_fwd_kernel(const NormParams p)
{
    constexpr int NT = 64 * NW;                            // threads of a row
    __shared__ float s_sum[ROWS][2][NW];
    const int t = threadIdx.x % NT, side = threadIdx.x / NT;
    RowSum<NW> sum = {s_sum[side], 0};
    constexpr bool HELD = NCH == 1;                        // weights and the next row stay in registers
    int cnt[NCH];
    float wpost[8], wres[8], wpre[8];
    const auto weights = [&](int j, bool after) {
        const int c = (j * NT + t) * LANE_CH;
        if (!after) {
            load_weight(p.post, c, cnt[j], 1.f, wpost);
            load_weight(p.res, c, cnt[j], 1.f, wres);
#pragma unroll
            for (int i = 0; i < 8; ++i) wres[i] *= p.scale;
        } else {
            load_weight(p.pre, c, cnt[j], 0.f, wpre);
        }
    };
#pragma unroll
    for (int j = 0; j < NCH; ++j) cnt[j] = max(0, min(LANE_CH, p.D - (j * NT + t) * LANE_CH));
    if (HELD) {
        weights(0, false);
        weights(0, true);
    }
    Raw8<X> xr[NCH];
    Raw8<T> yr[NCH], gr[NCH];
    const auto load = [&](int row) {
        const size_t r = min(row, p.R - 1);
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int c = (j * NT + t) * LANE_CH;
            xr[j].load((const X *)p.x.p + r * p.D + c, cnt[j]);
            if (p.y.p) yr[j].load((const T *)p.y.p + r * p.y.stride + c, cnt[j]);
            if (p.gate.p) gr[j].load((const T *)p.gate.p + r * p.gate.stride + c, cnt[j]);
        }
    };
    const float inv_d = 1.f / (float)p.D;
    const int step = gridDim.x * ROWS;
    if (HELD) load(blockIdx.x * ROWS + side);
    // all sides stay while one has a row: sums are joined behind barriers
    for (int row0 = blockIdx.x * ROWS; row0 < p.R; row0 += step) {
        const int row = row0 + side;
        const bool in = row < p.R;
        const size_t r = min(row, p.R - 1);
        if (!HELD) load(row);
        float x[NCH][8], u[NCH][8], g[NCH][8];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[j][i] = xr[j][i];
                if (p.y.p) u[j][i] = yr[j][i];
                if (p.gate.p) g[j][i] = gr[j][i];
            }
        if (HELD && row0 + step < p.R) load(row + step);
        if (p.y.p) {
            float rs = 1.f;
            if (p.post) {
#pragma unroll
                for (int j = 0; j < NCH; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss += u[j][i] * u[j][i];
                rs = rstd_of(sum(ss) * inv_d + p.eps);
            }
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = (j * NT + t) * LANE_CH, n = in ? cnt[j] : 0;
                if (p.y8.codes) store_codes<LANE_CH>(p.y8, r, p.D, c, n, u[j]);
                if (p.gate8.codes) store_codes<LANE_CH>(p.gate8, r, p.D, c, n, g[j]);
                if (!HELD) weights(j, false);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v = wpost[i] * (u[j][i] * rs);
                    if (p.gate.p) v *= sigmoid2(g[j][i]).s;
                    x[j][i] = to_f<X>(from_f<X>(x[j][i] + wres[i] * v));
                }
                if (n > 0) Raw8<X>::store((X *)p.x_out + r * p.D + c, n, x[j]);
            }
        }
        if (p.x8.codes)
#pragma unroll
            for (int j = 0; j < NCH; ++j)
                store_codes<LANE_CH>(p.x8, r, p.D, (j * NT + t) * LANE_CH, in ? cnt[j] : 0, x[j]);
        if (p.pre) {
            ss = 0.f;
#pragma unroll
            for (int j = 0; j < NCH; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss += x[j][i] * x[j][i];
            const float rs = rstd_of(sum(ss) * inv_d + p.eps);
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = (j * NT + t) * LANE_CH;
                if (!HELD) weights(j, true);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = wpre[i] * (x[j][i] * rs);
                if (in && cnt[j] > 0) Raw8<T>::store((T *)p.n + r * p.D + c, cnt[j], x[j]);
            }
        }
    }
}

// Four channels of a row's values, for the gradients: zeros (an open gate) where there is no such part.
struct Floats {
    float x[4], y[4], dx[4], dn[4];
    Sigmoid gate[4];
};

// Weights of channels [c, c + n): post, res times scale, pre.
__device__ __forceinline__ void load_weights(const NormParams &p, unsigned c, int n, f32x4 &post, f32x4 &res, f32x4 &pre)
{
    float w[3][4] = {{1.f, 1.f, 1.f, 1.f}, {1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}};
    if (p.post) load_f4(at_byte(p.post, 4 * c), n, w[0]);
    if (p.res) load_f4(at_byte(p.res, 4 * c), n, w[1]);
    if (p.pre) load_f4(at_byte(p.pre, 4 * c), n, w[2]);
    post = f32x4{w[0][0], w[0][1], w[0][2], w[0][3]};
    res = f32x4{w[1][0], w[1][1], w[1][2], w[1][3]} * p.scale;
    pre = f32x4{w[2][0], w[2][1], w[2][2], w[2][3]};
}

// Adds to the row's sums: y^2, x^2, w_pre dn x, A dx, A w_pre dn, A x.
__device__ __forceinline__ void add_sums(const Floats &f, f32x4 wpost, f32x4 wres, f32x4 wpre, float *s)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float d = wpre[i] * f.dn[i], A = wpost[i] * wres[i] * (f.y[i] * f.gate[i].s);
        s[0] += f.y[i] * f.y[i];
        s[1] += f.x[i] * f.x[i];
        s[2] += d * f.x[i];
        s[3] += A * f.dx[i];
        s[4] += A * d;
        s[5] += A * f.x[i];
    }
}

// 1 / rms of y and x', the means of w_pre dn x^ and of w_post du y^.
struct RowNumbers {
    float ry, rx, mx, my;
    __device__ __forceinline__ RowNumbers(const NormParams &p, bool pre, const float *s)
    {
        const float inv_d = 1.f / (float)p.D;
        ry = p.post ? rstd_of(s[0] * inv_d + p.eps) : 1.f;
        rx = pre ? rstd_of(s[1] * inv_d + p.eps) : 0.f;
        mx = s[2] * rx * inv_d;
        my = p.post ? (s[3] + rx * (s[4] - rx * mx * s[5])) * ry * inv_d : 0.f;
    }
    __device__ __forceinline__ explicit RowNumbers(f32x4 v) : ry(v[0]), rx(v[1]), mx(v[2]), my(v[3]) {}
};

// The gradients at four channels, and their parts of the weights' (res times scale at the end).
__device__ __forceinline__ void gradients(const Floats &f, const RowNumbers &k, f32x4 wpost, f32x4 wres, f32x4 wpre, f32x4 &post,
                                          f32x4 &res, f32x4 &pre, float *G, float *dy, float *dgate)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float xh = f.x[i] * k.rx, yh = f.y[i] * k.ry, u = wpost[i] * yh;
        pre[i] += f.dn[i] * xh;
        G[i] = f.dx[i] + k.rx * (wpre[i] * f.dn[i] - xh * k.mx);
        const float dr = G[i] * wres[i], du = dr * f.gate[i].s;
        res[i] += G[i] * (f.gate[i].s * u);
        post[i] += du * yh;
        dgate[i] = dr * u * (f.gate[i].s * f.gate[i].r);
        dy[i] = k.ry * (wpost[i] * du - yh * k.my);
    }
}

// Four or eight channels of a row of all that the gradients read, as it is stored.
template <typename T, typename X, int V> struct Values {
    HeldV<X, V> x, dx;
    HeldV<T, V> y, gate, dn;
    __device__ __forceinline__ void load(const NormParams &p, size_t r, unsigned c, unsigned from, int n)
    {
        if (p.y.p) y.load(p.y, r, p.D, c, from, n);
        if (p.pre && p.d_n) {
            x.load(p.x, r, p.D, c, from, n);
            dn.load({p.d_n, nullptr, p.D}, r, p.D, c, from, n);
        }
        if (p.d_x) dx.load({p.d_x, nullptr, p.D}, r, p.D, c, from, n);
        if (p.gate.p) gate.load(p.gate, r, p.D, c, from, n);
    }
    __device__ __forceinline__ void load(const NormParams &p, size_t r, unsigned c, int n) { load(p, r, c, c, n); }
    __device__ __forceinline__ void drop(const NormParams &p, int e)
    {
        if (p.y.p) y.drop(p.y.scales, e);
        if (p.pre && p.d_n) {
            x.drop(p.x.scales, e);
            dn.drop(false, e);
        }
        if (p.d_x) dx.drop(false, e);
        if (p.gate.p) gate.drop(p.gate.scales, e);
    }
    // Channels [4 k, 4 k + 4), or zeros.
    __device__ __forceinline__ void get(const NormParams &p, int k, bool in, Floats &f) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.x[i] = f.y[i] = f.dn[i] = f.dx[i] = 0.f;
            f.gate[i] = Sigmoid{1.f, 0.f};
        }
        if (!in) return;
        if (p.y.p) y.get(p.y.scales, k, f.y);
        if (p.gate.p) {
            float z[4];
            gate.get(p.gate.scales, k, z);
#pragma unroll
            for (int i = 0; i < 4; ++i) f.gate[i] = sigmoid2(z[i]);
        }
        if (p.pre && p.d_n) {
            x.get(p.x.scales, k, f.x);
            dn.get(false, k, f.dn);
        }
        if (p.d_x) dx.get(false, k, f.dx);
    }
    __device__ __forceinline__ void clear()
    {
        x.clear();
        y.clear();
        gate.clear();
        dx.clear();
        dn.clear();
    }
    __device__ __forceinline__ void hold()
    {
        x.hold();
        y.hold();
        gate.hold();
        dx.hold();
        dn.hold();
    }
};

// n of four channels' gradients.
template <typename T, typename X>
__device__ __forceinline__ void store_gradients(const NormParams &p, size_t r, unsigned c, int n, const float *G, const float *dy,
                                                const float *dgate)
{
    Raw4<X>::store(at_byte((X *)p.dx + r * p.D, c * sizeof(X)), n, G);
    if (p.y.p) Raw4<T>::store(at_byte((T *)p.dy + r * p.dy_stride, c * sizeof(T)), n, dy);
    if (p.gate.p) Raw4<T>::store(at_byte((T *)p.dgate + r * p.dgate_stride, c * sizeof(T)), n, dgate);
}

// A workgroup's sums of the weights' gradients.
__device__ __forceinline__ void store_sums(const NormParams &p, int part, unsigned c, int n, f32x4 post, f32x4 res, f32x4 pre)
{
    float *at = p.part + (size_t)part * p.D + c;
    const size_t other = (size_t)p.parts * p.D;
    const auto put = [&](f32x4 q, float *to) {
        const float v[4] = {q[0], q[1], q[2], q[3]};
        Raw4<float>::store(to, n, v);
    };
    if (p.dpost) put(post, at);
    if (p.dres) put(res, at + other);
    if (p.dpre) put(pre, at + 2 * other);
}

// Four floats a lane for each of NQ pieces: in registers, or in LDS, where a lane reads and writes its own places only.
template <int NT, int NQ, bool LDS> struct Quads;
template <int NT, int NQ> struct Quads<NT, NQ, false> {
    f32x4 v[NQ];
    __device__ __forceinline__ void begin(float *) {}
    __device__ __forceinline__ f32x4 get(int j) const { return v[j]; }
    __device__ __forceinline__ void put(int j, f32x4 x) { v[j] = x; }
};
template <int NT, int NQ> struct Quads<NT, NQ, true> {
    f32x4 *at;
    __device__ __forceinline__ void begin(float *lds) { at = reinterpret_cast<f32x4 *>(lds) + threadIdx.x; }
    __device__ __forceinline__ f32x4 get(int j) const { return at[j * NT]; }
    __device__ __forceinline__ void put(int j, f32x4 x) { at[j * NT] = x; }
};

// Gradients.  One sum over the row is enough: with A = w_post Sigmoid(gate) s y,
//   sum of w_post du y = sum A dx + rx sum A w_pre dn - rx^2 mx sum A x,
// so a row has one barrier between its two looks at the values (two: 160 us for 8192 x 4096 from 8 bits).  NW waves hold a row,
// NQ times 4 channels a lane.  With 4 (up to 4096 channels) the weights, their sums, a row and the next one as it is stored fit
// 128 registers, so that 16 waves a unit hide the sum: 98 to 105 us from 8 bits (439 MB, 4.2 TB/s or more) and 131 in bf16 (8 channels a lane and 8 waves:
// 143 us from 8 bits).  With 8 the weights lie in LDS, and the
// row's values are unpacked a second time for the second look.
// RAGGED: the last channels of a row are fewer than a lane's four.  The lane loads the row's last four all the same and takes those before
// its own off where it needs the values, since loads of single channels, each with its condition, wait for one another: 8192 x 4002
// 143 us instead of 198, 8192 x 4001 from 8 bits 119 instead of 186.  (A kernel that asks for either at run time takes 152 instead of
// 135 us for whole rows; with 8 channels a lane the same is slower, 201 us instead of 180 for 4096 x 8001: there the last lane
// goes by elements.)
template <typename T, typename X, int NW, int ROWS, int NQ, bool RAGGED>
__global__ __launch_bounds__(64 * NW * ROWS, 4) void norm_bwd_kernel(const NormParams p)
{
    constexpr int NT = 64 * NW, V = NQ == 1 ? 4 : 8;
    constexpr bool KEEP = NQ == 1;                         // numbers stay from look to look, the next row is on its way
    static_assert(NQ <= 2, "one piece of V channels a lane");
    extern __shared__ __align__(16) float s_mem[];         // NQ 2: weights [3][2][NT][4]; at the end [ROWS - 1][3][NT][4]
    __shared__ float s_sum[ROWS][2][NW][8];
    const int t = threadIdx.x % NT, side = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    RowSum6<NW> total = {s_sum[side], 0};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    // With D a multiple of V a lane has V channels or none, and asks nothing more; else the last one goes by elements.
    const bool whole = !RAGGED && p.D % V == 0;
    const int cnt = max(0, min(V, p.D - t * V));
    const bool ragged = RAGGED && __any(cnt > 0 && cnt < V);
    const auto channel = [&](int j) { return (unsigned)(t * V + 4 * j); };
    const auto count = [&](int j) { return max(0, min(4, p.D - (int)channel(j))); };
    Quads<NT, NQ, !KEEP> w_post, w_res, w_pre;
    f32x4 a_post[NQ], a_res[NQ], a_pre[NQ];
    w_post.begin(s_mem);
    w_res.begin(s_mem + 4 * NQ * NT);
    w_pre.begin(s_mem + 8 * NQ * NT);
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        f32x4 a, b, c;
        load_weights(p, channel(j), count(j), a, b, c);
        w_post.put(j, a);
        w_res.put(j, b);
        w_pre.put(j, c);
        a_post[j] = a_res[j] = a_pre[j] = zero;
    }
    Values<T, X, V> next;
    const auto load = [&](int row) {
        const size_t r = min(row, p.R - 1);
        if (RAGGED) {
            if (cnt > 0) next.load(p, r, t * V, min(t * V, p.D - V), V);
        } else if (whole) {
            if (cnt > 0) next.load(p, r, t * V, V);
        } else {
            next.load(p, r, t * V, cnt);
        }
    };
    next.clear();                                          // lanes without channels keep zeros
    int step = p.parts * ROWS, first = blockIdx.x * ROWS, end = p.R;
    if constexpr (ROWS > 1)
        // p.groups workgroups at a time go through a stretch of rows (all through all rows: 2^20 x 256 1100 us instead of 916)
        if (p.parts > p.groups) {
            step = p.groups * ROWS;
            const int stretch = step * NORM_CHAIN, turn = blockIdx.x / p.groups;
            first = turn * stretch + (blockIdx.x - turn * p.groups) * ROWS;
            end = (int)min((unsigned)p.R, (unsigned)(turn * stretch) + stretch);
        }
    if (KEEP) load(first + side);
    for (int row0 = first; row0 < end; row0 += step) {
        const int row = row0 + side;
        const bool in = ROWS == 1 || row < p.R;            // a side without a row adds zeros
        const size_t r = min(row, p.R - 1);
        if (!KEEP) load(row);
        Values<T, X, V> now = next;
        if constexpr (RAGGED)
            if (ragged) now.drop(p, cnt > 0 ? V - cnt : 0);
        if (KEEP && row0 + step < end) load(row + step);
        float s[6] = {};
        Floats f;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            now.get(p, j, in, f);
            add_sums(f, w_post.get(j), w_res.get(j), w_pre.get(j), s);
            if (!KEEP) __builtin_amdgcn_sched_barrier(0);
        }
        total(s);
        const RowNumbers k(p, p.pre && p.d_n, s);
        if (!KEEP) now.hold();
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int n = in ? count(j) : 0;
            if (!KEEP) now.get(p, j, in, f);
            float G[4], dy[4], dgate[4];
            gradients(f, k, w_post.get(j), w_res.get(j), w_pre.get(j), a_post[j], a_res[j], a_pre[j], G, dy, dgate);
            if (n > 0) {
                if (whole) store_gradients<T, X>(p, r, channel(j), 4, G, dy, dgate);
                else store_gradients<T, X>(p, r, channel(j), n, G, dy, dgate);
            }
            if (!KEEP) __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (ROWS > 1) {                                        // the sides' sums, in their order (NQ 1)
        f32x4 *at = reinterpret_cast<f32x4 *>(s_mem) + t;
        if (side > 0) {
            at[(side - 1) * 3 * NT] = a_post[0];
            at[((side - 1) * 3 + 1) * NT] = a_res[0];
            at[((side - 1) * 3 + 2) * NT] = a_pre[0];
        }
        __syncthreads();
        if (side > 0) return;
        for (int k = 0; k < ROWS - 1; ++k) {
            a_post[0] += at[k * 3 * NT];
            a_res[0] += at[(k * 3 + 1) * NT];
            a_pre[0] += at[(k * 3 + 2) * NT];
        }
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j)
        if (count(j) > 0) store_sums(p, blockIdx.x, channel(j), count(j), a_post[j], a_res[j] * p.scale, a_pre[j]);
}

// Rows of more than norm_row_d channels do not fit a workgroup's registers next to the weights and their sums (as one such kernel
// with the sums in LDS 2048 x 16384 took 447 us, 64 rows 130): a first kernel forms each row's numbers, a second goes
// through columns of 1024 channels with the weights and sums in registers and no barrier.  The values are read twice: 240 us, 3.2 TB/s
// with the second reading; 64 rows 33 us.
constexpr int WIDE_WAVES = 8;
template <typename T, typename X> __global__ __launch_bounds__(64 * WIDE_WAVES, 4) void norm_numbers_kernel(const NormParams p)
{
    constexpr int NT = 64 * WIDE_WAVES, BATCH = 4;         // pieces of 4 channels a lane on their way
    __shared__ float s_sum[2][WIDE_WAVES][8];
    RowSum6<WIDE_WAVES> total = {s_sum, 0};
    for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
        float s[6] = {};
        for (int c0 = 0; c0 < p.D; c0 += 4 * NT * BATCH) {
            Values<T, X, 4> v[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int c = c0 + 4 * (j * NT + (int)threadIdx.x);
                v[j].clear();
                if (c < p.D) v[j].load(p, r, c, min(4, p.D - c));
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int c = c0 + 4 * (j * NT + (int)threadIdx.x);
                f32x4 wpost, wres, wpre;
                Floats f;
                if (c < p.D) {
                    load_weights(p, c, min(4, p.D - c), wpost, wres, wpre);
                    v[j].get(p, 0, true, f);
                    add_sums(f, wpost, wres, wpre, s);
                }
            }
        }
        total(s);
        const RowNumbers k(p, p.pre && p.d_n, s);
        if (threadIdx.x == 0) p.numbers[r] = f32x4{k.ry, k.rx, k.mx, k.my};
    }
}
template <typename T, typename X> __global__ __launch_bounds__(256, 4) void norm_columns_kernel(const NormParams p)
{
    const int columns = (p.D + NORM_COLUMN - 1) / NORM_COLUMN, part = blockIdx.x / columns;
    const int c = (blockIdx.x % columns) * NORM_COLUMN + threadIdx.x * 4, n = max(0, min(4, p.D - c));
    if (n == 0) return;
    f32x4 wpost, wres, wpre, post = {0.f, 0.f, 0.f, 0.f}, res = post, pre = post;
    load_weights(p, c, n, wpost, wres, wpre);
    Values<T, X, 4> next;
    next.clear();
    if (part < p.R) next.load(p, part, c, n);
    for (int r = part; r < p.R; r += p.parts) {
        const Values<T, X, 4> now = next;
        const RowNumbers k(p.numbers[r]);
        if (r + p.parts < p.R) next.load(p, r + p.parts, c, n);
        Floats f;
        now.get(p, 0, true, f);
        float G[4], dy[4], dgate[4];
        gradients(f, k, wpost, wres, wpre, post, res, pre, G, dy, dgate);
        store_gradients<T, X>(p, r, c, n, G, dy, dgate);
    }
    store_sums(p, part, c, n, post, res * p.scale, pre);
}

// The weights' gradients from the workgroups' sums, in their order.  16 columns a workgroup (64 bytes of a row), SLICES threads down
// each, eight rows on their way: 7.4 us for 256 x 3 x 4096 sums (with 64 columns and 4 threads, one row at a time, 36 us
// for twice as many).  The many sums of very many rows, over few columns, take four times the threads: 4096 x 3 x 256 33 us (with 16
// threads 68).
template <int SLICES> __global__ __launch_bounds__(16 * SLICES) void norm_sum_kernel(const NormParams p)
{
    __shared__ double s_part[SLICES][16];
    float *out = blockIdx.y == 0 ? p.dpost : blockIdx.y == 1 ? p.dres : p.dpre;
    if (!out) return;
    const double sum = column_sum<SLICES>(p.part + (size_t)blockIdx.y * p.parts * p.D, p.parts, p.D, s_part);
    const int c = blockIdx.x * 16 + threadIdx.x;
    if (threadIdx.x < 16 && c < p.D) out[c] = (float)sum;
}

template <typename T, typename X, int NW, int ROWS, int NCH> static hipError_t launch_fwd_t(const NormParams &p, hipStream_t stream)
{
    const int grid = (p.R + ROWS - 1) / ROWS, most = 256 * 16 / (NW * ROWS);         // 16 waves on each of 256 units
    hipLaunchKernelGGL((norm_fwd_kernel<T, X, NW, ROWS, NCH>), dim3(grid < most ? grid : most), dim3(64 * NW * ROWS), 0, stream, p);
    return hipGetLastError();
}

static hipError_t launch_sum(const NormParams &p, hipStream_t stream)
{
    if (p.dpost || p.dres || p.dpre) {
        const dim3 grid((p.D + 15) / 16, 3);
        if (p.parts > 1024)
            hipLaunchKernelGGL((norm_sum_kernel<64>), grid, dim3(1024), 0, stream, p);
        else
            hipLaunchKernelGGL((norm_sum_kernel<16>), grid, dim3(256), 0, stream, p);
    }
    return hipGetLastError();
}

template <typename T, typename X> static hipError_t launch_bwd_wide(const NormParams &p, hipStream_t stream)
{
    if (p.R > 0) {
        const int most = 256 * 4;                                                    // two a unit at a time, in two turns
        hipLaunchKernelGGL((norm_numbers_kernel<T, X>), dim3(p.R < most ? p.R : most), dim3(64 * WIDE_WAVES), 0, stream, p);
        hipLaunchKernelGGL((norm_columns_kernel<T, X>), dim3(p.parts * ((p.D + NORM_COLUMN - 1) / NORM_COLUMN)), dim3(256), 0, stream, p);
    }
    return launch_sum(p, stream);
}

template <typename T, typename X, int NW, int ROWS, int NQ> static hipError_t launch_bwd_t(const NormParams &p, hipStream_t stream)
{
    static_assert(NW * ROWS == norm_waves(256 * NW * NQ) && ROWS == norm_rows(256 * NW * NQ), "as planned");
    constexpr size_t row = sizeof(float) * 256 * NW * NQ;                            // of floats
    constexpr size_t lds = row * (NQ == 1 ? 3 * (ROWS - 1) : 3);
    if (p.R > 0) {
        const auto kernel = NQ == 1 && p.D % 4 != 0 && p.D > 4 ? norm_bwd_kernel<T, X, NW, ROWS, NQ, NQ == 1>
                                                                  : norm_bwd_kernel<T, X, NW, ROWS, NQ, false>;
        if (lds > 0) {
            const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(kernel, dim3(p.parts), dim3(64 * NW * ROWS), lds, stream, p);
    }
    return launch_sum(p, stream);
}

// Forward: 8 channels a lane, as few waves a row as that takes, up to 16; then twice the channels.  Fewer lanes without channels,
// and sums over fewer waves: 2^25 elements in rows of 512, 1024, 2048, 4096, 8192 channels take 61 to 63 us; as the next
// wider form 77 to 78, of 8192 channels 108.
template <typename T, typename X> static hipError_t launch_fwd_x(const NormParams &p, hipStream_t stream)
{
    if (p.D <= 512) return launch_fwd_t<T, X, 1, 4, 1>(p, stream);
    if (p.D <= 1024) return launch_fwd_t<T, X, 2, 2, 1>(p, stream);
    if (p.D <= 2048) return launch_fwd_t<T, X, 4, 1, 1>(p, stream);
    if (p.D <= 4096) return launch_fwd_t<T, X, 8, 1, 1>(p, stream);
    if (p.D <= 8192) return launch_fwd_t<T, X, 16, 1, 1>(p, stream);
    return launch_fwd_t<T, X, 16, 1, 2>(p, stream);
}

// Backward: 4 channels a lane, as few waves a row as that takes, up to 16; then more channels.  2^25 elements of bf16 in rows of 256
// to 8192 channels take 138 to 146 us; as the next wider form 217 to 228 (up to 1024 channels), 192 (2048), 177 (4096).
template <typename T, typename X> static hipError_t launch_bwd_x(const NormParams &p, hipStream_t stream)
{
    if (p.D <= 256) return launch_bwd_t<T, X, 1, 4, 1>(p, stream);
    if (p.D <= 512) return launch_bwd_t<T, X, 2, 2, 1>(p, stream);
    if (p.D <= 1024) return launch_bwd_t<T, X, 4, 1, 1>(p, stream);
    if (p.D <= 2048) return launch_bwd_t<T, X, 8, 1, 1>(p, stream);
    if (p.D <= 4096) return launch_bwd_t<T, X, 16, 1, 1>(p, stream);
    if constexpr (norm_row_d(sizeof(T) == 4) > 4096)
        if (p.D <= norm_row_d(sizeof(T) == 4)) return launch_bwd_t<T, X, 16, 1, 2>(p, stream);
    return launch_bwd_wide<T, X>(p, stream);
}

hipError_t launch_norm_fwd(int is_bf16, int x_bf16, const NormParams &p, hipStream_t stream)
{
    if (!is_bf16) return launch_fwd_x<float, float>(p, stream);
    return x_bf16 ? launch_fwd_x<bf16, bf16>(p, stream) : launch_fwd_x<bf16, float>(p, stream);
}

hipError_t launch_norm_bwd(int is_bf16, int x_bf16, const NormParams &p, hipStream_t stream)
{
    if (!is_bf16) return launch_bwd_x<float, float>(p, stream);
    return x_bf16 ? launch_bwd_x<bf16, bf16>(p, stream) : launch_bwd_x<bf16, float>(p, stream);
}

}  // namespace kda
