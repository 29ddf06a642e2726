// balance.cu -- balance loss, z-loss and per-expert counts over the sequences of
// a ragged, padded batch, with the gradient of the routing logits.
//
// A token counts where seq_starts[i] <= t < seq_starts[i+1] for a sequence i and
// its mask byte is not zero.  With n_i counted tokens in sequence i, S' sequences
// that have some and N counted tokens in all,
//   counts[i,e] = #{(t,k) : t counts in i, ids[t,k] = e},  f[i,e] = counts / (n_i K)
//   L_i = E sum_e f[i,e] (1/n_i) sum_t p[t,e] = (E / n_i) sum_t c_t,  c_t = sum_e f[i,e] p[t,e]
//   balance = (1/S') sum_i L_i,   z = (1/N) sum_t lse_t^2
//   d logits[t,:] = c_balance E / (S' n_i) dp[t,:] (f[i,:] - c_t) + c_z 2 lse_t / N softmax[t,:]
// (counts carry no gradient; dp = p for the softmax, p (1 - sigmoid) for sigmoid
// scores).  The sum over tokens of c_t is all the loss needs, so the mean
// probabilities are never formed, and the logits are read once: the counts, which
// the gradient needs first, come from the ids alone.
//
// Sums do not depend on the order of the blocks: counts are integers; a
// sequence's c_t, each in [0, 1], are added as integers of 2^-32 (half a step,
// 2^-33, is far below fp32's own rounding of a c_t near 1/E >= 2^-8); z is summed
// per block in fp64 and the blocks' sums are added in order by the last block.
#include "internal.h"
#include "common.cuh"

namespace moe {

constexpr int kBalTokens = 32;     // tokens per block of the gradient pass (8 warps)
constexpr int kBalPerLane = 8;     // experts per lane: E <= 256
constexpr double kBalFix = 4294967296.0;  // 2^32

MOE_DEVICE float bal_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
MOE_DEVICE float bal_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Scratch of a call, laid out by balance_layout.
struct BalScratch {
    int* status;
    int* done;                // blocks that have finished
    int* used;                // S': sequences with a counted token
    unsigned long long* all;  // N: counted tokens
    int* tokens;              // (S) n_i
    int* bad;                 // (S) a counted token's c_t is not a number
    unsigned long long* acc;  // (S) sum of c_t in 2^-32
    double* zpart;            // per block: sum of lse^2
};

struct BalArgs {
    const float* logits;
    const int32_t* ids;
    const int32_t* starts;
    const uint8_t* mask;
    int32_t* counts;
    float* losses;
    float* seq_loss;
    float* dlogits;
    int64_t T;
    int E, K, S, sigmoid;
    float c_balance, c_z;
    BalScratch w;
};

// The sequence a token counts in, or -1.
MOE_DEVICE int bal_sequence(const BalArgs& a, int64_t t)
{
    int lo = 0, hi = a.S;  // largest i with starts[i] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)a.starts[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    if (lo >= a.S || (int64_t)a.starts[lo] > t || (int64_t)a.starts[lo + 1] <= t) return -1;
    return a.mask == nullptr || a.mask[t] != 0 ? lo : -1;
}

__global__ void __launch_bounds__(256) balance_zero_kernel(BalArgs a)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * 256;
    if (i == 0) {
        *a.w.done = 0;
        *a.w.used = 0;
        *a.w.all = 0;
    }
    for (int64_t k = i; k < a.S; k += step) {
        a.w.tokens[k] = 0;
        a.w.bad[k] = 0;
        a.w.acc[k] = 0;
        const int64_t b0 = a.starts[k], b1 = a.starts[k + 1];
        if (b0 < 0 || b1 < b0 || b1 > a.T) raise_flag(a.w.status, kFlagBounds, 710);
    }
    for (int64_t k = i; k < (int64_t)a.S * a.E; k += step) a.counts[k] = 0;
}

__global__ void __launch_bounds__(256) balance_count_kernel(BalArgs a)
{
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= a.T) return;
    const int i = bal_sequence(a, t);
    if (i < 0) return;
    if (atomicAdd(&a.w.tokens[i], 1) == 0) atomicAdd(a.w.used, 1);
    atomicAdd(a.w.all, 1ull);
    for (int k = 0; k < a.K; ++k) {
        const int id = a.ids[t * a.K + k];
        if (id < 0 || id >= a.E) raise_flag(a.w.status, kFlagBounds, 711);
        else atomicAdd(&a.counts[(int64_t)i * a.E + id], 1);
    }
}

__global__ void __launch_bounds__(256) balance_grad_kernel(BalArgs a)
{
    __shared__ double zs[8];
    __shared__ int last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E;
    const float total = (float)*a.w.all, used = (float)*a.w.used;
    double z = 0.0;
    for (int n = 0; n < kBalTokens / 8; ++n) {
        const int64_t t = (int64_t)blockIdx.x * kBalTokens + n * 8 + warp;
        if (t >= a.T) break;
        const int i = bal_sequence(a, t);
        float* out = a.dlogits != nullptr ? a.dlogits + t * E : nullptr;
        if (i < 0) {
            if (out != nullptr)
                for (int e = lane; e < E; e += 32) out[e] = 0.f;
            continue;
        }
        const float* L = a.logits + t * E;
        float l[kBalPerLane], p[kBalPerLane];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < kBalPerLane; ++j) {
            const int e = lane + 32 * j;
            l[j] = e < E ? L[e] : -INFINITY;
            mx = fmaxf(mx, l[j]);
        }
        mx = bal_max(mx);
        float se = 0.f, sg = 0.f;
#pragma unroll
        for (int j = 0; j < kBalPerLane; ++j) {
            const bool in = lane + 32 * j < E;
            p[j] = in ? expf(l[j] - mx) : 0.f;
            se += p[j];
            if (a.sigmoid) {
                l[j] = in ? 1.f / (1.f + expf(-l[j])) : 0.f;  // the score
                sg += l[j];
            }
        }
        se = bal_sum(se);
        if (a.sigmoid) sg = bal_sum(sg);
        const float lse = mx + logf(se);
        const float inv_n = 1.f / (float)a.w.tokens[i];
        const float fscale = inv_n / (float)a.K;
        const int32_t* cnt = a.counts + (int64_t)i * E;
        float f[kBalPerLane], c = 0.f;
#pragma unroll
        for (int j = 0; j < kBalPerLane; ++j) {
            const int e = lane + 32 * j;
            f[j] = e < E ? (float)cnt[e] * fscale : 0.f;
            c += f[j] * (a.sigmoid ? l[j] / sg : p[j] / se);
        }
        c = bal_sum(c);
        z += (double)lse * (double)lse;
        if (lane == 0) {
            if (c >= 0.f && c <= 1.5f)
                atomicAdd(&a.w.acc[i], (unsigned long long)((double)c * kBalFix + 0.5));
            else
                a.w.bad[i] = 1;
        }
        if (out != nullptr) {
            const float cb = a.c_balance * (float)E / used * inv_n, cz = a.c_z * 2.f * lse / total;
#pragma unroll
            for (int j = 0; j < kBalPerLane; ++j) {
                const int e = lane + 32 * j;
                if (e >= E) continue;
                const float soft = p[j] / se;
                const float dp = a.sigmoid ? l[j] / sg * (1.f - l[j]) : soft;
                out[e] = cb * dp * (f[j] - c) + cz * soft;
            }
        }
    }
    if (lane == 0) zs[warp] = z;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < 8; ++w) s += zs[w];
        a.w.zpart[blockIdx.x] = s;
        __threadfence();
        last = atomicAdd(a.w.done, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // the block that finishes last: per-sequence losses, then both means
    __shared__ double red[2][256];
    double zsum = 0.0, bsum = 0.0;
    for (int64_t b = threadIdx.x; b < gridDim.x; b += 256) zsum += __ldcg(&a.w.zpart[b]);
    for (int64_t i = threadIdx.x; i < a.S; i += 256) {
        const int n = __ldcg(&a.w.tokens[i]);
        double L = 0.0;
        if (n > 0)
            L = __ldcg(&a.w.bad[i]) ? (double)NAN : (double)E * ((double)__ldcg(&a.w.acc[i]) / kBalFix) / (double)n;
        a.seq_loss[i] = (float)L;
        bsum += L;
    }
    red[0][threadIdx.x] = zsum;
    red[1][threadIdx.x] = bsum;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if ((int)threadIdx.x < o) {
            red[0][threadIdx.x] += red[0][threadIdx.x + o];
            red[1][threadIdx.x] += red[1][threadIdx.x + o];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const unsigned long long all = __ldcg(a.w.all);
        const int u = __ldcg(a.w.used);
        a.losses[0] = all ? (float)(red[0][0] / (double)all) : 0.f;
        a.losses[1] = u ? (float)(red[1][0] / (double)u) : 0.f;
    }
}

// ------------------------------------------------------------------- host --
struct BalLayout {
    size_t head, tokens, bad, acc, zpart, total;
};
static int64_t bal_blocks(const moe_config& c) { return (c.T + kBalTokens - 1) / kBalTokens; }
static BalLayout balance_layout(const moe_config& c, int64_t S)
{
    BalLayout L;
    size_t o = 0;
    L.head = o;   o += 256;  // status word, then at 64 bytes the call's counters
    L.tokens = o; o += align_up((size_t)S * 4);
    L.bad = o;    o += align_up((size_t)S * 4);
    L.acc = o;    o += align_up((size_t)S * 8);
    L.zpart = o;  o += align_up((size_t)bal_blocks(c) * 8);
    L.total = o;
    return L;
}
size_t balance_bytes(const moe_config& c, int64_t S) { return balance_layout(c, S).total; }

cudaError_t launch_balance(const moe_config& c, int64_t S, const float* logits, const int32_t* ids,
                           const int32_t* starts, const uint8_t* mask, float c_balance, float c_z, int32_t* counts,
                           float* losses, float* seq_loss, float* dlogits, void* ws, cudaStream_t s)
{
    const BalLayout L = balance_layout(c, S);
    char* w = static_cast<char*>(ws);
    BalArgs a;
    a.logits = logits; a.ids = ids; a.starts = starts; a.mask = mask;
    a.counts = counts; a.losses = losses; a.seq_loss = seq_loss; a.dlogits = dlogits;
    a.T = c.T; a.E = c.E; a.K = c.K; a.S = (int)S; a.sigmoid = c.score_func == MOE_SCORE_SIGMOID;
    a.c_balance = c_balance; a.c_z = c_z;
    a.w.status = reinterpret_cast<int*>(w + L.head);
    a.w.done = reinterpret_cast<int*>(w + L.head + 64);
    a.w.used = reinterpret_cast<int*>(w + L.head + 68);
    a.w.all = reinterpret_cast<unsigned long long*>(w + L.head + 72);
    a.w.tokens = reinterpret_cast<int*>(w + L.tokens);
    a.w.bad = reinterpret_cast<int*>(w + L.bad);
    a.w.acc = reinterpret_cast<unsigned long long*>(w + L.acc);
    a.w.zpart = reinterpret_cast<double*>(w + L.zpart);
    int64_t zb = (S * c.E + 255) / 256;
    if (zb > 148) zb = 148;
    balance_zero_kernel<<<(unsigned)zb, 256, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    balance_count_kernel<<<(unsigned)((c.T + 255) / 256), 256, 0, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    balance_grad_kernel<<<(unsigned)bal_blocks(c), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
