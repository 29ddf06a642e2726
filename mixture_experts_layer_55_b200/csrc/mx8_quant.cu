// mx8_quant.cu -- into and out of 8-bit blocks (mx8.cuh): rows of activations,
// weights laid out for the 8-bit experts, and the values back.
//
// All three are one pass over the data, bound by HBM.
#include "internal.h"
#include "mx8.cuh"

namespace moe {

template <typename T> MOE_DEVICE void load8v(const T* p, float (&v)[8]);
template <> MOE_DEVICE void load8v<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8])
{
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <> MOE_DEVICE void load8v<float>(const float* p, float (&v)[8])
{
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// n elements in blocks of 32; a block is four neighbouring lanes of 8 elements.
template <typename T>
__global__ void __launch_bounds__(256) mx8_quantize_kernel(const T* x, uint8_t* q, uint8_t* scales, int64_t nvec)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    float v[8];
    uint32_t m = 0;
    const bool in = i < nvec;  // nvec is a multiple of 4: a block's lanes agree
    if (in) {
        load8v<T>(x + 8 * i, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (!in) return;
    const uint32_t b = mx_scale_byte(m);
    const float inv = mx_inv_scale(b);
    *reinterpret_cast<uint2*>(q + 8 * i) =
        make_uint2(mx_pack4(v[0], v[1], v[2], v[3], inv), mx_pack4(v[4], v[5], v[6], v[7], inv));
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
}

// The values: e4m3 times its power of two, exact in fp32 and (four significant
// bits) in bf16 down to the type's own least values.
template <typename T>
__global__ void __launch_bounds__(256) mx8_dequantize_kernel(const uint8_t* q, const uint8_t* scales, T* out,
                                                             int64_t nvec)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= nvec) return;
    const uint2 w = *reinterpret_cast<const uint2*>(q + 8 * i);
    const float sc = mx_scale(scales[i >> 2]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = e4m3_to_f32((w.x >> (8 * j)) & 0xffu) * sc;
        v[4 + j] = e4m3_to_f32((w.y >> (8 * j)) & 0xffu) * sc;
    }
    if (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(out + 8 * i) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
        float4* o = reinterpret_cast<float4*>(out + 8 * i);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// w (E, K, N) -> q (E, N, K), scales (E, N, K / 32): the contracted axis becomes
// the contiguous one.  A thread owns one column and one block of 32: its reads
// are coalesced over the columns, its 32 bytes are one whole sector.
template <typename T>
__global__ void __launch_bounds__(128) mx8_weight_kernel(const T* w, uint8_t* q, uint8_t* scales, int K, int N)
{
    const int n = (int)(blockIdx.x * 128 + threadIdx.x);
    if (n >= N) return;
    const int kb = (int)blockIdx.y;
    const int64_t e = blockIdx.z;
    const T* src = w + (e * K + (int64_t)kb * kMxBlock) * N + n;
    float v[kMxBlock];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
        v[i] = to_f32<T>(src[(int64_t)i * N]);
        m = max(m, abs_bits(v[i]));
    }
    const uint32_t b = mx_scale_byte(m);
    const float inv = mx_inv_scale(b);
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = mx_pack4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], inv);
    uint4* dst = reinterpret_cast<uint4*>(q + (e * N + n) * K + (int64_t)kb * kMxBlock);
    dst[0] = make_uint4(p[0], p[1], p[2], p[3]);
    dst[1] = make_uint4(p[4], p[5], p[6], p[7]);
    scales[(e * N + n) * (K / kMxBlock) + kb] = (uint8_t)b;
}

// Rows of 8-bit tokens and their scales to their expert-major places:
// xq_perm[row] = xq[perm[row] / K] for row < offsets[E].  One warp per row.
__global__ void __launch_bounds__(256)
    mx8_gather_kernel(const uint8_t* xq, const uint8_t* xs, const int32_t* offsets, const int32_t* perm,
                      uint8_t* xq_perm, uint8_t* xs_perm, int D, int E, int K, int64_t T, int64_t max_rows,
                      int* status)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t rows = offsets[E];
    if (row >= rows || row >= max_rows) return;
    const int32_t p = perm[row];
    const int64_t t = p / K;
    if (p < 0 || t >= T) {
        if (lane == 0) raise_flag(status, kFlagBounds, 700);
        return;
    }
    const uint4* src = reinterpret_cast<const uint4*>(xq + t * D);
    uint4* dst = reinterpret_cast<uint4*>(xq_perm + row * D);
    for (int i = lane; i < D / 16; i += 32) dst[i] = src[i];
    const int nb = D / kMxBlock;
    for (int i = lane; i < nb; i += 32) xs_perm[row * nb + i] = xs[t * nb + i];
}

// ------------------------------------------------------------------- host --
cudaError_t launch_mx8_quantize(int64_t n, int dtype, const void* x, void* q, void* scales, cudaStream_t s)
{
    const int64_t nvec = n / 8;
    const unsigned grid = (unsigned)((nvec + 255) / 256);
    uint8_t *pq = static_cast<uint8_t*>(q), *ps = static_cast<uint8_t*>(scales);
    if (dtype == MOE_BF16)
        mx8_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), pq, ps, nvec);
    else
        mx8_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(x), pq, ps, nvec);
    return cudaGetLastError();
}

cudaError_t launch_mx8_dequantize(int64_t n, int dtype, const void* q, const void* scales, void* out,
                                  cudaStream_t s)
{
    const int64_t nvec = n / 8;
    const unsigned grid = (unsigned)((nvec + 255) / 256);
    const uint8_t *pq = static_cast<const uint8_t*>(q), *ps = static_cast<const uint8_t*>(scales);
    if (dtype == MOE_BF16)
        mx8_dequantize_kernel<<<grid, 256, 0, s>>>(pq, ps, static_cast<__nv_bfloat16*>(out), nvec);
    else
        mx8_dequantize_kernel<<<grid, 256, 0, s>>>(pq, ps, static_cast<float*>(out), nvec);
    return cudaGetLastError();
}

cudaError_t launch_mx8_weight(int E, int K, int N, int dtype, const void* w, void* q, void* scales, cudaStream_t s)
{
    const dim3 grid((unsigned)((N + 127) / 128), (unsigned)(K / kMxBlock), (unsigned)E);
    uint8_t *pq = static_cast<uint8_t*>(q), *ps = static_cast<uint8_t*>(scales);
    if (dtype == MOE_BF16)
        mx8_weight_kernel<<<grid, 128, 0, s>>>(static_cast<const __nv_bfloat16*>(w), pq, ps, K, N);
    else
        mx8_weight_kernel<<<grid, 128, 0, s>>>(static_cast<const float*>(w), pq, ps, K, N);
    return cudaGetLastError();
}

cudaError_t launch_mx8_gather(const moe_config& c, const void* xq, const void* xs, const int32_t* offsets,
                              const int32_t* perm, void* xq_perm, void* xs_perm, int64_t max_rows, int* status,
                              cudaStream_t s)
{
    mx8_gather_kernel<<<(unsigned)((max_rows + 7) / 8), 256, 0, s>>>(
        static_cast<const uint8_t*>(xq), static_cast<const uint8_t*>(xs), offsets, perm,
        static_cast<uint8_t*>(xq_perm), static_cast<uint8_t*>(xs_perm), c.D, c.E, c.K, c.T, max_rows, status);
    return cudaGetLastError();
}

}  // namespace moe
