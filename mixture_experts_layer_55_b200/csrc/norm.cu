// norm.cu -- residual addition and root-mean-square norm before the layer, its
// 8-bit output, and its backward.
//
//   s = x + residual, rounded to the layer dtype (it is stored and carried on;
//       the norm is that of the stored sum)
//   r = (mean_d s^2 + eps)^(-1/2)                       fp32
//   n = s r gamma, rounded to the layer dtype
//   q, scales = n in 8-bit blocks of 32 (mx8.cuh)
// and, with xh = s r and g = dn gamma,
//   dx = ds + r (g - xh mean_d(g xh)),   dgamma = sum_t dn xh.
//
// Bound: HBM.  A row is read once into registers (8 elements per 16- or 32-byte
// vector, VPT vectors per thread, consecutive lanes on consecutive vectors), so
// every array crosses memory once; the squares and dot products are summed in
// fp32 in an order fixed by the shape.  A block of 32 elements is four
// neighbouring lanes: its maximum takes two shuffles.
#include "internal.h"
#include "mx8.cuh"

namespace moe {

constexpr int kNormMaxThreads = 1024;

// Eight elements as they lie in memory, and as fp32.
template <typename T> struct Row8;
template <> struct Row8<__nv_bfloat16> {
    struct Raw { uint4 q; };
    MOE_DEVICE static Raw fetch(const __nv_bfloat16* p) { return {*reinterpret_cast<const uint4*>(p)}; }
    MOE_DEVICE static void values(const Raw& r, float (&v)[8])
    {
        const uint32_t w[4] = {r.q.x, r.q.y, r.q.z, r.q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // stores v rounded to bf16 and leaves the rounded values in v
    MOE_DEVICE static void store(__nv_bfloat16* p, float (&v)[8])
    {
        Raw r;
        r.q = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
        if (p != nullptr) *reinterpret_cast<uint4*>(p) = r.q;
        values(r, v);
    }
};
template <> struct Row8<float> {
    struct Raw { float4 a, b; };
    MOE_DEVICE static Raw fetch(const float* p)
    {
        return {reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
    }
    MOE_DEVICE static void values(const Raw& r, float (&v)[8])
    {
        v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
        v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
    }
    MOE_DEVICE static void store(float* p, float (&v)[8])
    {
        if (p == nullptr) return;
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <typename T> MOE_DEVICE void load_row8(const T* p, float (&v)[8]) { Row8<T>::values(Row8<T>::fetch(p), v); }

MOE_DEVICE float warp_add(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the `warps` warps of a row (one warp: no barrier).  red: one slot per
// warp; every thread adds the slots in order.  The caller alternates two slot
// arrays, so that one barrier per sum is enough.
MOE_DEVICE float row_add(float v, float* red, int warps)
{
    v = warp_add(v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < warps; ++w) t += red[w];
    return t;
}

struct NormArgs {
    int64_t T;
    int D, nvec;     // nvec = D / 8
    int warps;       // warps per row
    float eps;
    const float* gamma;
    float* rstd;     // (T) or null
    uint8_t* q;      // (T, D) or null
    uint8_t* scales; // (T, D / 32)
};

// A team of `warps` warps (a block, or with warps = 1 each warp of it) walks
// rows and loads the next row while it reduces and writes one.  x, residual, s
// and n may be the same memory: a thread reads its elements of a row before it
// writes them, and no other thread touches them.
template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_kernel(const T* x, const T* residual, T* s_out, T* n_out,
                                                                  const NormArgs a)
{
    __shared__ float red[2][32];
    using R = Row8<T>;
    const int tpr = a.warps * 32;
    const int teams = a.warps == 1 ? (int)(blockDim.x >> 5) : 1;
    const int64_t team = a.warps == 1 ? (int64_t)blockIdx.x * teams + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * teams;
    const int tid = a.warps == 1 ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    typename R::Raw rx[VPT], rr[VPT];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            if (c < a.nvec) {
                rx[i] = R::fetch(x + row * a.D + 8 * c);
                if (residual != nullptr) rr[i] = R::fetch(residual + row * a.D + 8 * c);
            }
        }
    };
    constexpr bool AHEAD = VPT * MAXT <= 1024;  // wider rows need the registers
    if (AHEAD && team < a.T) fetch(team);
    int flip = 0;
    for (int64_t row = team; row < a.T; row += step, flip ^= 1) {
        const int64_t base = row * a.D;
        if (!AHEAD) fetch(row);
        float v[VPT][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            if (c < a.nvec) {
                R::values(rx[i], v[i]);
                if (residual != nullptr) {
                    float r[8];
                    R::values(rr[i], r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] += r[j];
                    R::store(s_out != nullptr ? s_out + base + 8 * c : nullptr, v[i]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
            }
        }
        if (AHEAD && row + step < a.T) fetch(row + step);
        ss = row_add(ss, red[flip], a.warps);
        const float r = 1.0f / sqrtf(ss / (float)a.D + a.eps);
        if (tid == 0 && a.rstd != nullptr) a.rstd[row] = r;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            const bool in = c < a.nvec;
            if (in) {
                float g[8];
                load_row8<float>(a.gamma + 8 * c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * g[j];
                R::store(n_out != nullptr ? n_out + base + 8 * c : nullptr, v[i]);
            }
            if (a.q != nullptr) {
                uint32_t m = 0;
                if (in)
#pragma unroll
                    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));  // nvec is a multiple of 4:
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));  // a block's lanes are all in or all out
                if (in) {
                    const uint32_t b = mx_scale_byte(m);
                    const float inv = mx_inv_scale(b);
                    *reinterpret_cast<uint2*>(a.q + base + 8 * c) =
                        make_uint2(mx_pack4(v[i][0], v[i][1], v[i][2], v[i][3], inv),
                                   mx_pack4(v[i][4], v[i][5], v[i][6], v[i][7], inv));
                    if ((c & 3) == 0) a.scales[row * (a.D / kMxBlock) + (c >> 2)] = (uint8_t)b;
                }
            }
        }
    }
}

struct NormBwdArgs {
    int64_t T;
    int D, nvec, warps;
    const float* gamma;
    const float* rstd;
    float* part;  // (gridDim.x * rows per block, D): each row team's share of dgamma
};

// A team of `warps` warps walks rows; each thread keeps its columns' share of
// dgamma in registers and writes it once, so dn and s cross memory once.
template <typename T, int VPT>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_backward_kernel(const T* dn, const T* ds, const T* s, T* dx, const NormBwdArgs a)
{
    __shared__ float red[2][32];
    const int tpr = a.warps * 32;
    const int teams = a.warps == 1 ? (int)(blockDim.x >> 5) : 1;
    const int64_t team = a.warps == 1 ? (int64_t)blockIdx.x * teams + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * teams;
    const int tid = a.warps == 1 ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    using R = Row8<T>;
    float acc[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    typename R::Raw rs[VPT], rn[VPT], rd[VPT];
    float r_next = 0.f;
    auto fetch = [&](int64_t row) {  // the next row, while one is reduced and written
        r_next = a.rstd[row];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            if (c < a.nvec) {
                rs[i] = R::fetch(s + row * a.D + 8 * c);
                rn[i] = R::fetch(dn + row * a.D + 8 * c);
                if (ds != nullptr) rd[i] = R::fetch(ds + row * a.D + 8 * c);
            }
        }
    };
    constexpr bool AHEAD = VPT == 1;  // wider rows need the registers
    if (AHEAD && team < a.T) fetch(team);
    int flip = 0;
    for (int64_t row = team; row < a.T; row += step, flip ^= 1) {
        const int64_t base = row * a.D;
        if (!AHEAD) fetch(row);
        const float r = r_next;
        float xh[VPT][8], g[VPT][8];
        typename R::Raw d0[VPT];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            if (c < a.nvec) {
                float w[8];
                R::values(rs[i], xh[i]);
                R::values(rn[i], g[i]);
                d0[i] = rd[i];
                load_row8<float>(a.gamma + 8 * c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[i][j] *= r;
                    acc[i][j] = fmaf(g[i][j], xh[i][j], acc[i][j]);
                    g[i][j] *= w[j];
                    dot = fmaf(g[i][j], xh[i][j], dot);
                }
            }
        }
        if (AHEAD && row + step < a.T) fetch(row + step);
        dot = row_add(dot, red[flip], a.warps) / (float)a.D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            if (c < a.nvec) {
                float o[8];
                if (ds != nullptr) R::values(d0[i], o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = r * (g[i][j] - xh[i][j] * dot);
                    o[j] = ds != nullptr ? d + o[j] : d;
                }
                R::store(dx + base + 8 * c, o);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        if (c < a.nvec) Row8<float>::store(a.part + team * a.D + 8 * c, acc[i]);
    }
}

// dgamma[d] = sum of the teams' shares: 8 warps per 32 columns, each with every
// 8th team, then added in order.
__global__ void __launch_bounds__(256) rmsnorm_dgamma_kernel(const float* part, int teams, int D, float* dgamma)
{
    __shared__ float sum[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int d = (int)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (d < D) {
#pragma unroll 8
        for (int p = w; p < teams; p += 8) t += part[(int64_t)p * D + d];
    }
    sum[w][lane] = t;
    __syncthreads();
    if (w == 0 && d < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) t += sum[i][lane];
        dgamma[d] = t;
    }
}

// ------------------------------------------------------------------- host --
// Vectors per thread and warps per row.  Few rows (fewer than four per SM) want
// the shortest path, a vector per thread; many want loads in flight, up to four
// vectors in 256 threads (T = 8192, D = 4096 bf16 with a residual: 43.6 us, 0.94 of
// the measured copy bandwidth, against 47.2 with a vector in each of 512
// threads; T = 128, D = 7168: 3.7 us with 896 threads, 4.4 with 256).
struct NormPlan {
    int vpt, warps, threads, rows_per_block;
};
static NormPlan norm_plan(int D, int most_threads)
{
    NormPlan p;
    const int nvec = D / 8;
    p.vpt = 1;
    while (p.vpt < 8 && (nvec + p.vpt - 1) / p.vpt > most_threads) p.vpt *= 2;
    p.warps = ((nvec + p.vpt - 1) / p.vpt + 31) / 32;
    p.threads = p.warps == 1 ? 128 : p.warps * 32;
    p.rows_per_block = p.warps == 1 ? 4 : 1;
    return p;
}

template <typename T>
static cudaError_t launch_norm_t(int64_t rows, int D, const void* x, const void* residual, void* s_out,
                                 void* n_out, const NormArgs& a, const NormPlan& p, cudaStream_t s)
{
    const int64_t need = (rows + p.rows_per_block - 1) / p.rows_per_block;
    const int64_t most = 148 * (int64_t)(2048 / p.threads);
    const unsigned grid = (unsigned)(need < most ? need : most);
    const T *px = static_cast<const T*>(x), *pr = static_cast<const T*>(residual);
    T *ps = static_cast<T*>(s_out), *pn = static_cast<T*>(n_out);
    if (p.threads <= 256 && p.vpt == 2) rmsnorm_kernel<T, 2, 256><<<grid, p.threads, 0, s>>>(px, pr, ps, pn, a);
    else if (p.threads <= 256 && p.vpt == 4) rmsnorm_kernel<T, 4, 256><<<grid, p.threads, 0, s>>>(px, pr, ps, pn, a);
    else if (p.vpt == 1) rmsnorm_kernel<T, 1, 1024><<<grid, p.threads, 0, s>>>(px, pr, ps, pn, a);
    else if (p.vpt == 2) rmsnorm_kernel<T, 2, 1024><<<grid, p.threads, 0, s>>>(px, pr, ps, pn, a);
    else if (p.vpt == 4) rmsnorm_kernel<T, 4, 1024><<<grid, p.threads, 0, s>>>(px, pr, ps, pn, a);
    else rmsnorm_kernel<T, 8, 1024><<<grid, p.threads, 0, s>>>(px, pr, ps, pn, a);
    return cudaGetLastError();
}

cudaError_t launch_rmsnorm(int64_t T, int D, int dtype, const void* x, const void* residual, const float* gamma,
                           float eps, void* s_out, void* n_out, float* rstd, void* q, void* scales,
                           cudaStream_t s)
{
    const NormPlan p = norm_plan(D, T >= 4 * 148 && D <= 8192 ? 256 : kNormMaxThreads);
    const NormArgs a{T, D, D / 8, p.warps, eps, gamma, rstd, static_cast<uint8_t*>(q), static_cast<uint8_t*>(scales)};
    return dtype == MOE_BF16 ? launch_norm_t<__nv_bfloat16>(T, D, x, residual, s_out, n_out, a, p, s)
                             : launch_norm_t<float>(T, D, x, residual, s_out, n_out, a, p, s);
}

// Row teams of the backward, a function of the shape alone (the workspace holds
// one row of dgamma for each).
static int64_t norm_bwd_blocks(int64_t T, const NormPlan& p)
{
    const int64_t need = (T + p.rows_per_block - 1) / p.rows_per_block;
    const int64_t most = 148 * 2;
    return need < most ? need : most;
}

size_t rmsnorm_backward_bytes(int64_t T, int D)
{
    const NormPlan p = norm_plan(D, kNormMaxThreads);
    return 256 + align_up((size_t)norm_bwd_blocks(T, p) * p.rows_per_block * D * sizeof(float));
}

template <typename T>
static void launch_norm_bwd_t(unsigned grid, const void* dn, const void* ds, const void* s_in, void* dx,
                              const NormBwdArgs& a, const NormPlan& p, cudaStream_t s)
{
    const T *pd = static_cast<const T*>(dn), *pe = static_cast<const T*>(ds), *ps = static_cast<const T*>(s_in);
    T* px = static_cast<T*>(dx);
    switch (p.vpt) {
    case 1: rmsnorm_backward_kernel<T, 1><<<grid, p.threads, 0, s>>>(pd, pe, ps, px, a); break;
    case 2: rmsnorm_backward_kernel<T, 2><<<grid, p.threads, 0, s>>>(pd, pe, ps, px, a); break;
    case 4: rmsnorm_backward_kernel<T, 4><<<grid, p.threads, 0, s>>>(pd, pe, ps, px, a); break;
    default: rmsnorm_backward_kernel<T, 8><<<grid, p.threads, 0, s>>>(pd, pe, ps, px, a); break;
    }
}

cudaError_t launch_rmsnorm_backward(int64_t T, int D, int dtype, const void* dn, const void* ds, const void* s_in,
                                    const float* gamma, const float* rstd, void* dx, float* dgamma, void* ws,
                                    cudaStream_t s)
{
    const NormPlan p = norm_plan(D, kNormMaxThreads);
    const int64_t blocks = norm_bwd_blocks(T, p);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
    const NormBwdArgs a{T, D, D / 8, p.warps, gamma, rstd, part};
    if (dtype == MOE_BF16) launch_norm_bwd_t<__nv_bfloat16>((unsigned)blocks, dn, ds, s_in, dx, a, p, s);
    else launch_norm_bwd_t<float>((unsigned)blocks, dn, ds, s_in, dx, a, p, s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    rmsnorm_dgamma_kernel<<<(D + 31) / 32, 256, 0, s>>>(part, (int)(blocks * p.rows_per_block), D, dgamma);
    return cudaGetLastError();
}

}  // namespace moe
