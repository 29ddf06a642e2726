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

// These kernels are launched while the one before them in the stream still ends
// (43.1 us of work took 46.6 in a row of plain launches, 44.6 so) and wait for it
// here, before they touch memory.
MOE_DEVICE void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
static cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                                const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

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

// The same with the warps' sums (a thread's at most 64 squares and five additions
// in fp32) added in fp64.
MOE_DEVICE double row_add_wide(float v, float* red, int warps)
{
    v = warp_add(v);
    if (warps == 1) return (double)v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < warps; ++w) t += (double)red[w];
    return t;
}

struct NormArgs {
    int64_t T;
    int D, nvec;     // nvec = D / 8
    int warps;       // warps per row
    float eps;
    double inv_d;    // 1 / D
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
    wait_for_stream();
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
    constexpr bool AHEAD = VPT * MAXT * (int)sizeof(T) <= 4096;  // else the registers are needed
    if (AHEAD && team < a.T) fetch(team);
    // a row's values times rstd stay below sqrt(D): their products with this thread's
    // weights are finite where the weights are below 2^100
    bool gamma_fits = true;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        if (c < a.nvec) {
            float g[8];
            load_row8<float>(a.gamma + 8 * c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) gamma_fits = gamma_fits && fabsf(g[j]) < 0x1p100f;
        }
    }
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
        double sum = row_add_wide(ss, red[flip], a.warps);
        double eps = a.eps;
        float half = 1.f;
        if (!(sum < 0x1p100) || (sum < 0x1p-90 && a.eps < 0x1p-100f)) {
            // the squares leave fp32 (or the row holds a NaN): again in units of 2^100 or
            // 2^-70, the whole team together.  The values and the root keep one half of the
            // unit each, so that both are normal numbers from fp32's least value to its
            // largest; eps in these units, up to 2^100, is formed in fp64.
            half = sum < 1.0 ? 0x1p50f : 0x1p-35f;
            eps *= ((double)half * half) * ((double)half * half);
            float again = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (tid + i * tpr < a.nvec)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[i][j] *= half;
                        const float u = v[i][j] * half;
                        again = fmaf(u, u, again);
                    }
            if (a.warps > 1) __syncthreads();  // the first sum's slots have been read
            sum = row_add_wide(again, red[flip], a.warps);
        }
        // rstd as the sum of two fp32 values, from fp32's root and one Newton step in
        // fp64: n is then the formula's rounded to fp32 but for a percent of cases, and
        // what is rounded further, to bf16 and to 8 bits, falls on the formula's side
        // of a border (the step in fp32 took the same time and missed a third).
        const double mean = sum * a.inv_d + eps;
        const float root = rsqrtf((float)mean);
        const double fine = (double)root * (1.5 - 0.5 * mean * (double)root * (double)root);
        // (not where the root says it all: a row of zeros without eps, an overflow, a
        // NaN; nor where r0's parts leave fp32)
        const bool carry = gamma_fits && root > 0x1p-60f && root < 0x1p60f;
        const float near = carry ? (float)fine : root;
        const float r0 = near * half, r_lo = carry ? (float)(fine - (double)near) * half : 0.f, r = r0 * half;
        if (tid == 0 && a.rstd != nullptr) a.rstd[row] = r;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            const bool in = c < a.nvec;
            if (in) {
                float g[8];
                load_row8<float>(a.gamma + 8 * c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {  // v r g with its roundings' errors carried along
                    const float t = v[i][j] * r0, n = t * g[j];
                    if (!carry) {
                        v[i][j] = n;
                        continue;
                    }
                    const float et = fmaf(v[i][j], r_lo, fmaf(v[i][j], r0, -t));
                    v[i][j] = n + fmaf(et, g[j], fmaf(t, g[j], -n));
                }
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
    float* part;  // (gridDim.x, D): each block's share of dgamma
};

// A team of `warps` warps (a block, or with warps = 1 each of its warps) walks
// rows; each thread keeps its columns' share of dgamma in registers and the block
// writes its share once, so dn and s cross memory once.  Where a thread has more
// than one vector the row is held as it was loaded and widened twice, before and
// after its sum (held in fp32, D = 12288 took 211 us for 2048 rows, spilled; 57 so);
// the next row is on its way meanwhile.  T = 8192, D = 4096
// bf16: 48.9 us with dgamma, 0.84 of the measured copy bandwidth.
template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_backward_kernel(const T* dn, const T* ds, const T* s, T* dx,
                                                                const NormBwdArgs a)
{
    __shared__ float red[2][32];
    extern __shared__ float share[];  // (warps of the block, D) where each warp has rows of its own
    using R = Row8<T>;
    const int tpr = a.warps * 32;
    const int teams = a.warps == 1 ? (int)(blockDim.x >> 5) : 1;
    const int64_t team = a.warps == 1 ? (int64_t)blockIdx.x * teams + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * teams;
    const int tid = a.warps == 1 ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    constexpr bool AHEAD = VPT * MAXT * (int)sizeof(T) <= 2048;  // else the registers are needed
    constexpr bool KEEP = VPT == 1 && sizeof(T) == 2;  // the widened row fits the registers
    float acc[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    wait_for_stream();
    typename R::Raw rs[VPT], rn[VPT], rd[VPT];
    float r_next = 0.f;
    auto fetch = [&](int64_t row) {
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
    if (AHEAD && team < a.T) fetch(team);
    int flip = 0;
    for (int64_t row = team; row < a.T; row += step, flip ^= 1) {
        const int64_t base = row * a.D;
        if (!AHEAD) fetch(row);
        const float r = r_next;
        typename R::Raw cs[VPT], cn[VPT], cd[VPT];
        float xk[KEEP ? VPT : 1][8], gk[KEEP ? VPT : 1][8];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            cs[i] = rs[i];
            cn[i] = rn[i];
            cd[i] = rd[i];
            if (c < a.nvec) {
                float xh[8], g[8], w[8];
                R::values(cs[i], xh);
                R::values(cn[i], g);
                load_row8<float>(a.gamma + 8 * c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[j] *= r;
                    acc[i][j] = fmaf(g[j], xh[j], acc[i][j]);
                    g[j] *= w[j];
                    dot = fmaf(g[j], xh[j], dot);
                    if (KEEP) {
                        xk[KEEP ? i : 0][j] = xh[j];
                        gk[KEEP ? i : 0][j] = g[j];
                    }
                }
            }
        }
        if (AHEAD && row + step < a.T) fetch(row + step);
        dot = row_add(dot, red[flip], a.warps) / (float)a.D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            if (c < a.nvec) {
                float xh[8], g[8], w[8], o[8];
                if (!KEEP) {
                    R::values(cs[i], xh);
                    R::values(cn[i], g);
                    load_row8<float>(a.gamma + 8 * c, w);
                }
                if (ds != nullptr) R::values(cd[i], o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (KEEP) {
                        xh[j] = xk[KEEP ? i : 0][j];
                        g[j] = gk[KEEP ? i : 0][j];
                    } else {
                        xh[j] *= r;
                        g[j] *= w[j];
                    }
                    const float d = r * (g[j] - xh[j] * dot);
                    o[j] = ds != nullptr ? d + o[j] : d;
                }
                R::store(dx + base + 8 * c, o);
            }
        }
    }
    if (a.warps == 1) {  // the block's warps add up first
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = tid + i * tpr;
            if (c < a.nvec) Row8<float>::store(share + (threadIdx.x >> 5) * a.D + 8 * c, acc[i]);
        }
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
            float t = 0.f;
            for (int w = 0; w < teams; ++w) t += share[w * a.D + d];
            a.part[(int64_t)blockIdx.x * a.D + d] = t;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        if (c < a.nvec) Row8<float>::store(a.part + (int64_t)blockIdx.x * a.D + 8 * c, acc[i]);
    }
}

// dgamma[d] = sum of the blocks' shares: 8 warps per 32 columns, each with every
// 8th block, then added in order.
__global__ void __launch_bounds__(256) rmsnorm_dgamma_kernel(const float* part, int teams, int D, float* dgamma)
{
    __shared__ float sum[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int d = (int)blockIdx.x * 32 + lane;
    float t = 0.f;
    wait_for_stream();
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

// One wave: as many row teams as are resident at once (T = 8192, D = 4096: 46.2 us
// with a third more blocks than that).
template <typename T, int VPT, int MAXT>
static cudaError_t launch_norm_v(int64_t rows, const T* x, const T* residual, T* s_out, T* n_out, const NormArgs& a,
                                 const NormPlan& p, cudaStream_t s)
{
    static std::atomic<int> cached[33];  // resident blocks per SM, by warps in a block (0: not yet asked)
    auto kernel = rmsnorm_kernel<T, VPT, MAXT>;
    const int w = p.threads / 32;
    int per_sm = cached[w].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, p.threads, 0);
        if (e != cudaSuccess) return e;
        if (per_sm < 1) return cudaErrorInvalidConfiguration;
        cached[w].store(per_sm, std::memory_order_relaxed);
    }
    const int64_t need = (rows + p.rows_per_block - 1) / p.rows_per_block, most = 148 * (int64_t)per_sm;
    return launch_early(kernel, (unsigned)(need < most ? need : most), (unsigned)p.threads, 0, s, x, residual, s_out,
                        n_out, a);
}

template <typename T>
static cudaError_t launch_norm_t(int64_t rows, const void* x, const void* residual, void* s_out, void* n_out,
                                 const NormArgs& a, const NormPlan& p, cudaStream_t s)
{
    const T *px = static_cast<const T*>(x), *pr = static_cast<const T*>(residual);
    T *ps = static_cast<T*>(s_out), *pn = static_cast<T*>(n_out);
    if (p.vpt == 1) return launch_norm_v<T, 1, 1024>(rows, px, pr, ps, pn, a, p, s);
    if (p.threads <= 256 && p.vpt == 2) return launch_norm_v<T, 2, 256>(rows, px, pr, ps, pn, a, p, s);
    if (p.threads <= 256 && p.vpt == 4) return launch_norm_v<T, 4, 256>(rows, px, pr, ps, pn, a, p, s);
    if (p.threads <= 512 && p.vpt == 4) return launch_norm_v<T, 4, 512>(rows, px, pr, ps, pn, a, p, s);
    if (p.vpt == 2) return launch_norm_v<T, 2, 1024>(rows, px, pr, ps, pn, a, p, s);
    if (p.vpt == 4) return launch_norm_v<T, 4, 1024>(rows, px, pr, ps, pn, a, p, s);
    return launch_norm_v<T, 8, 1024>(rows, px, pr, ps, pn, a, p, s);
}

cudaError_t launch_rmsnorm(int64_t T, int D, int dtype, const void* x, const void* residual, const float* gamma,
                           float eps, void* s_out, void* n_out, float* rstd, void* q, void* scales,
                           cudaStream_t s)
{
    const NormPlan p = norm_plan(D, T < 4 * 148 ? kNormMaxThreads : D <= 8192 ? 256 : 512);
    const NormArgs a{T, D, D / 8, p.warps, eps, 1.0 / D, gamma, rstd, static_cast<uint8_t*>(q), static_cast<uint8_t*>(scales)};
    return dtype == MOE_BF16 ? launch_norm_t<__nv_bfloat16>(T, x, residual, s_out, n_out, a, p, s)
                             : launch_norm_t<float>(T, x, residual, s_out, n_out, a, p, s);
}

// The backward: up to 1024 elements a warp has rows of its own (eight warps a
// block); wider rows are a block's, 512 threads of up to four vectors, and beyond
// 16384 elements 1024 threads.
static NormPlan norm_bwd_plan(int D)
{
    if (D > 1024) return norm_plan(D, D <= 16384 ? 512 : kNormMaxThreads);
    NormPlan p;
    p.vpt = D <= 256 ? 1 : D <= 512 ? 2 : 4;
    p.warps = 1;
    p.threads = 256;
    p.rows_per_block = 8;
    return p;
}

// Its blocks, a function of the shape alone (the workspace holds one row of dgamma
// for each).
static int64_t norm_bwd_blocks(int64_t T, const NormPlan& p)
{
    const int64_t need = (T + p.rows_per_block - 1) / p.rows_per_block;
    const int64_t most = 148 * (p.threads > 512 ? 1 : p.threads > 256 ? 2 : 4);
    return need < most ? need : most;
}

size_t rmsnorm_backward_bytes(int64_t T, int D)
{
    return 256 + align_up((size_t)norm_bwd_blocks(T, norm_bwd_plan(D)) * D * sizeof(float));
}

// *blocks: in, the most the workspace holds; out, the blocks launched (one wave).
template <typename T, int VPT, int MAXT>
static cudaError_t launch_norm_bwd_v(int64_t* blocks, const T* dn, const T* ds, const T* s_in, T* dx,
                                     const NormBwdArgs& a, const NormPlan& p, cudaStream_t s)
{
    const size_t smem = p.warps == 1 ? (size_t)p.rows_per_block * a.D * sizeof(float) : 0;  // at most 32 KB
    static std::atomic<int> cached[33];  // resident blocks per SM, by warps in a block (0: not yet asked)
    auto kernel = rmsnorm_backward_kernel<T, VPT, MAXT>;
    const int w = p.threads / 32;
    int per_sm = cached[w].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, p.threads,
                                                                      p.warps == 1 ? VPT * 256 * 8 * sizeof(float) : 0);
        if (e != cudaSuccess) return e;
        if (per_sm < 1) return cudaErrorInvalidConfiguration;
        cached[w].store(per_sm, std::memory_order_relaxed);
    }
    if (*blocks > 148 * (int64_t)per_sm) *blocks = 148 * (int64_t)per_sm;
    return launch_early(kernel, (unsigned)*blocks, (unsigned)p.threads, smem, s, dn, ds, s_in, dx, a);
}

template <typename T>
static cudaError_t launch_norm_bwd_t(int64_t* blocks, const void* dn, const void* ds, const void* s_in, void* dx,
                                     const NormBwdArgs& a, const NormPlan& p, cudaStream_t s)
{
    const T *pd = static_cast<const T*>(dn), *pe = static_cast<const T*>(ds), *ps = static_cast<const T*>(s_in);
    T* px = static_cast<T*>(dx);
    if (p.warps == 1) {
        if (p.vpt == 1) return launch_norm_bwd_v<T, 1, 256>(blocks, pd, pe, ps, px, a, p, s);
        if (p.vpt == 2) return launch_norm_bwd_v<T, 2, 256>(blocks, pd, pe, ps, px, a, p, s);
        return launch_norm_bwd_v<T, 4, 256>(blocks, pd, pe, ps, px, a, p, s);
    }
    if (p.threads <= 512) {
        if (p.vpt == 1) return launch_norm_bwd_v<T, 1, 512>(blocks, pd, pe, ps, px, a, p, s);
        if (p.vpt == 2) return launch_norm_bwd_v<T, 2, 512>(blocks, pd, pe, ps, px, a, p, s);
        return launch_norm_bwd_v<T, 4, 512>(blocks, pd, pe, ps, px, a, p, s);
    }
    if (p.vpt <= 4) return launch_norm_bwd_v<T, 4, 1024>(blocks, pd, pe, ps, px, a, p, s);
    return launch_norm_bwd_v<T, 8, 1024>(blocks, pd, pe, ps, px, a, p, s);
}

cudaError_t launch_rmsnorm_backward(int64_t T, int D, int dtype, const void* dn, const void* ds, const void* s_in,
                                    const float* gamma, const float* rstd, void* dx, float* dgamma, void* ws,
                                    cudaStream_t s)
{
    const NormPlan p = norm_bwd_plan(D);
    int64_t blocks = norm_bwd_blocks(T, p);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
    const NormBwdArgs a{T, D, D / 8, p.warps, gamma, rstd, part};
    cudaError_t e = dtype == MOE_BF16 ? launch_norm_bwd_t<__nv_bfloat16>(&blocks, dn, ds, s_in, dx, a, p, s)
                                      : launch_norm_bwd_t<float>(&blocks, dn, ds, s_in, dx, a, p, s);
    if (e != cudaSuccess) return e;
    return launch_early(rmsnorm_dgamma_kernel, (unsigned)((D + 31) / 32), 256, 0, s, (const float*)part, (int)blocks, D,
                        dgamma);
}

}  // namespace moe
