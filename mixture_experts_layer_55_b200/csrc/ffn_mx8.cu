// ffn_mx8.cu -- grouped SwiGLU experts on 8-bit rows and weights.
//
// Rows and weights are e4m3 in blocks of 32 along the contracted axis with
// power-of-two scales (mx8.cuh); for every row r of expert e
//   g = x_r . Wg_e,  u = x_r . Wu_e                       (K = D, fp32 sums)
//   h_r = 8-bit blocks of silu(g) u                       (blocks of 32 along F)
//   y_r = bf16(w_r (h_r . Wd_e))                          (K = F)
// h is rounded to 8 bits straight from fp32: at most 2^-4 of a value, the
// precision of every operand of these products.
//
// A simple kernel: 64 rows by 32 columns per block, the operands' values in
// shared memory in fp32, 32 of the contracted axis at a time.
#include "internal.h"
#include "mx8.cuh"

namespace moe {

constexpr int kSM = 64, kSN = 32;

struct Mx8Args {
    const int32_t* offsets;
    const int32_t* perm;
    const float* topk_w;
    const uint8_t *a, *as;    // (rows, Kdim), (rows, Kdim / 32)
    const uint8_t *b0, *b0s;  // (E, N, Kdim), (E, N, Kdim / 32): gate, or down
    const uint8_t *b1, *b1s;  // up
    uint8_t *h, *hs;          // gate/up: (rows, N), (rows, N / 32)
    __nv_bfloat16* y;         // down: (rows, N)
    int E, N, Kdim;
    int64_t max_rows, nk;
    int* status;
};

template <bool GATEUP> __global__ void __launch_bounds__(256) ffn_mx8_simple_kernel(Mx8Args a)
{
    __shared__ float sa[kSM][33], sb[GATEUP ? 2 : 1][kSN][33];
    // the expert and rows of this block's tile
    int e = 0, r0 = 0, r1 = 0;
    int64_t m = blockIdx.y;
    for (; e < a.E; ++e) {
        r0 = a.offsets[e];
        r1 = a.offsets[e + 1];
        if (r0 < 0 || r1 < r0 || r1 > a.max_rows) {
            if (threadIdx.x == 0) raise_flag(a.status, kFlagBounds, 720);
            return;
        }
        const int64_t tiles = (r1 - r0 + kSM - 1) / kSM;
        if (m < tiles) break;
        m -= tiles;
    }
    if (e == a.E) return;
    r0 += (int)m * kSM;
    const int n0 = blockIdx.x * kSN;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;  // column, group of 8 rows
    const int nb = a.Kdim / kMxBlock;
    float c0[8], c1[8];
    for (int i = 0; i < 8; ++i) c0[i] = c1[i] = 0.f;
    for (int kb = 0; kb < nb; ++kb) {
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + ty * 8 + i;
            sa[ty * 8 + i][tx] =
                r < r1 ? e4m3_to_f32(a.a[(int64_t)r * a.Kdim + kb * 32 + tx]) * mx_scale(a.as[(int64_t)r * nb + kb])
                       : 0.f;
        }
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + ty * 4 + i;
            const int64_t row = (int64_t)e * a.N + n;
            sb[0][ty * 4 + i][tx] =
                n < a.N ? e4m3_to_f32(a.b0[row * a.Kdim + kb * 32 + tx]) * mx_scale(a.b0s[row * nb + kb]) : 0.f;
            if (GATEUP)
                sb[GATEUP ? 1 : 0][ty * 4 + i][tx] =
                    n < a.N ? e4m3_to_f32(a.b1[row * a.Kdim + kb * 32 + tx]) * mx_scale(a.b1s[row * nb + kb]) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < 32; ++k)
            for (int i = 0; i < 8; ++i) {
                c0[i] = fmaf(sa[ty * 8 + i][k], sb[0][tx][k], c0[i]);
                if (GATEUP) c1[i] = fmaf(sa[ty * 8 + i][k], sb[GATEUP ? 1 : 0][tx][k], c1[i]);
            }
        __syncthreads();
    }
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + ty * 8 + i;  // uniform in the warp
        if (r >= r1) break;
        if (GATEUP) {
            const float h = silu_f32(c0[i]) * c1[i];
            const uint32_t mx = __reduce_max_sync(0xffffffffu, abs_bits(h));
            const uint32_t b = mx_scale_byte(mx);
            a.h[(int64_t)r * a.N + n0 + tx] = (uint8_t)(mx_pack4(h, 0.f, 0.f, 0.f, mx_inv_scale(b)) & 0xffu);
            if (tx == 0) a.hs[(int64_t)r * (a.N / 32) + n0 / 32] = (uint8_t)b;
        } else if (n0 + tx < a.N) {
            float w = 1.f;
            if (a.perm != nullptr) {
                const int32_t p = a.perm[r];
                if (p >= 0 && (int64_t)p < a.nk) w = a.topk_w[p];
                else { raise_flag(a.status, kFlagBounds, 721); w = 0.f; }
            }
            a.y[(int64_t)r * a.N + n0 + tx] = __float2bfloat16_rn(w * c0[i]);
        }
    }
}

// ------------------------------------------------------------------- host --
cudaError_t launch_ffn_mx8(const moe_config& c, int64_t max_rows, const void* xq, const void* xs,
                           const int32_t* offsets, const int32_t* perm, const float* topk_w,
                           const moe_mx8_weights& w, void* hq, void* hs, void* y_perm, int* status, cudaStream_t s)
{
    auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
    const unsigned mt = (unsigned)((max_rows + kSM - 1) / kSM + c.E);
    Mx8Args a{};
    a.offsets = offsets; a.perm = perm; a.topk_w = topk_w;
    a.a = u8(xq); a.as = u8(xs);
    a.b0 = u8(w.gate); a.b0s = u8(w.gate_scales); a.b1 = u8(w.up); a.b1s = u8(w.up_scales);
    a.h = static_cast<uint8_t*>(hq); a.hs = static_cast<uint8_t*>(hs);
    a.E = c.E; a.N = c.F; a.Kdim = c.D; a.max_rows = max_rows; a.nk = c.T * c.K; a.status = status;
    ffn_mx8_simple_kernel<true><<<dim3((c.F + kSN - 1) / kSN, mt), 256, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    a.a = u8(hq); a.as = u8(hs);
    a.b0 = u8(w.down); a.b0s = u8(w.down_scales);
    a.y = static_cast<__nv_bfloat16*>(y_perm);
    a.N = c.D; a.Kdim = c.F;
    ffn_mx8_simple_kernel<false><<<dim3((c.D + kSN - 1) / kSN, mt), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
