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
// sequence's c_t, each in [0, 1], are added as integers of 2^-(63 - b), b the bits
// of T, the finest unit whose sum over T tokens cannot overflow.  A c_t, an fp32
// number, is held exactly from 2^(b - 40) on, and to half a unit below: seq_loss
// is off by at most E 2^-(64 - b).  z is summed per thread and block in fp64 and the
// blocks' sums are added in order by the block that finishes last.
//
// One cooperative launch (every block resident): zero the results, count, and the
// gradient, with two grid barriers between them.  Both are split: a block
// arrives, does what does not depend on the others (its histogram in shared
// memory; its first tokens' softmax), and then waits.  A block takes consecutive
// tokens, a token a group of L lanes with 8 experts each, so that a warp is full
// for 8 experts as for 256.  Bound: latency (launch, two barriers, a handful of
// dependent loads) up to a few megabytes of logits, then the instructions of a
// token's softmax.  Measured (with the gradient; in us): T = 8192, E = 8, 4
// sequences 10.4; T = 32768, E = 256, 16 sequences 25.9 (its logits and gradient
// take 10.2 at the measured copy bandwidth); T = 16384, E = 64, sigmoid, 37
// sequences 15.7.  The first two as three launches, with a warp per token: 30 and 64.
#include "internal.h"
#include "common.cuh"

namespace moe {

constexpr int kBalThreads = 256;
constexpr int kBalMaxBlocks = 444;  // 3 per SM
constexpr int kBalPer = 8;          // experts per lane: E <= 256
constexpr int kBalStarts = 2048;    // sequence borders held in shared memory, else searched in global
constexpr int kBalHist = 4096;      // (sequence, expert) counters of a block's tokens
constexpr int kBalSpan = 512;       // and sequences

// Scratch of a call, laid out by balance_layout.
struct BalScratch {
    int* status;              // flags
    uint32_t* bar;            // grid barrier: arrivals (zero between calls)
    uint32_t* done;           // blocks that have finished (zero between calls)
    int* tokens;              // (S) n_i
    int* bad;                 // (S) a counted token's c_t is not a number
    unsigned long long* acc;  // (S) sum of c_t in units of 1 / fix
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
    int64_t T, chunk;  // tokens, tokens per block
    int E, K, S;
    float c_balance, c_z;
    float fix;          // 2^(63 - b), T < 2^b
    BalScratch w;
};

struct BalShared {
    int starts[kBalStarts];
    int hist[kBalHist];
    int tokens[kBalSpan];
    double red[2][kBalThreads / 32];
    unsigned long long all[kBalThreads / 32];
    int used[kBalThreads / 32];
    int lo, hi, last;
};

// Largest i in 0 .. S with starts[i] <= t (0 when there is none).
MOE_DEVICE int bal_find(const int32_t* starts, int S, int64_t t)
{
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)starts[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The sequence a token counts in, or -1.
MOE_DEVICE int bal_sequence(const BalArgs& a, const int32_t* starts, int64_t t)
{
    const int i = bal_find(starts, a.S, t);
    if (i >= a.S || (int64_t)starts[i] > t || (int64_t)starts[i + 1] <= t) return -1;
    return a.mask == nullptr || a.mask[t] != 0 ? i : -1;
}

// The grid barrier in two halves: a count of arrivals that only grows within a
// call (the block that finishes last sets it back to zero).  Thread 0's release
// covers what the block's other threads wrote before the block barrier.
MOE_DEVICE void bal_arrive(const BalArgs& a)
{
    __syncthreads();
    if (threadIdx.x == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.w.bar) : "memory");
}

// Waits for the n-th arrival of every block.  Bounded: after kWaitLimitNs the
// timeout flag is raised and the block goes on (its results are then flagged as
// invalid).
MOE_DEVICE void bal_wait(const BalArgs& a, uint32_t n)
{
    if (threadIdx.x == 0) {
        uint32_t spins = 0, v;
        uint64_t t0 = 0;
        while (true) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.w.bar) : "memory");
            if (v >= n * gridDim.x) break;
            if ((++spins & 1023u) == 0u) {
                if (t0 == 0) t0 = globaltimer_ns();
                else if (globaltimer_ns() - t0 > kWaitLimitNs) {
                    raise_flag(a.w.status, kFlagTimeout, 712);
                    break;
                }
            }
        }
    }
    __syncthreads();
}

// Reads of what other blocks have written in this launch: the compiler keeps them
// behind the wait that they follow.
MOE_DEVICE int bal_read(const int* p)
{
    int v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
MOE_DEVICE unsigned long long bal_read(const unsigned long long* p)
{
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
MOE_DEVICE double bal_read(const double* p)
{
    double v;
    asm volatile("ld.relaxed.gpu.global.f64 %0, [%1];" : "=d"(v) : "l"(p) : "memory");
    return v;
}
MOE_DEVICE int4 bal_read(const int4* p)
{
    int4 v;
    asm volatile("ld.relaxed.gpu.global.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

template <int L> MOE_DEVICE float group_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int L> MOE_DEVICE float group_max(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A lane's experts: 8 consecutive ones (rows of a multiple of 4: two 16-byte
// vectors), or every L-th; of the logits, or of a row of counts, which this launch
// writes.
MOE_DEVICE int4 bal_get4(const float* p) { return __ldcg(reinterpret_cast<const int4*>(p)); }
MOE_DEVICE int4 bal_get4(const int* p) { return bal_read(reinterpret_cast<const int4*>(p)); }
MOE_DEVICE float bal_get(const float* p) { return __ldcg(p); }
MOE_DEVICE int bal_get(const int* p) { return bal_read(p); }

template <int L, bool VEC, typename V>
MOE_DEVICE void bal_load(const V* row, int lg, int E, V (&v)[kBalPer], V pad)
{
    if (VEC) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int e = lg * kBalPer + 4 * q;
            if (e < E) {
                const int4 w = bal_get4(row + e);
                const int x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * q + i] = *reinterpret_cast<const V*>(&x[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * q + i] = pad;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) {
            const int e = lg + L * j;
            v[j] = e < E ? bal_get(row + e) : pad;
        }
    }
}

template <int L, bool VEC>
MOE_DEVICE void bal_store(float* row, int lg, int E, const float (&v)[kBalPer])
{
    if (VEC) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int e = lg * kBalPer + 4 * q;
            if (e < E)
                *reinterpret_cast<float4*>(row + e) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) {
            const int e = lg + L * j;
            if (e < E) row[e] = v[j];
        }
    }
}

template <int L, bool VEC, bool SIG> __global__ void __launch_bounds__(kBalThreads, 3) balance_kernel(const BalArgs a)
{
    __shared__ BalShared sh;
    const int tid = threadIdx.x, E = a.E;
    const int64_t gtid = (int64_t)blockIdx.x * kBalThreads + tid, gstep = (int64_t)gridDim.x * kBalThreads;
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = t0 + a.chunk < a.T ? t0 + a.chunk : a.T;
    int first_id[8];  // the ids of the thread's first token (K <= 8), on their way from here
#pragma unroll
    for (int k = 0; k < 8; ++k) first_id[k] = t0 + tid < t1 && k < a.K ? a.ids[(t0 + tid) * a.K + k] : 0;
    // zero this call's sums, then check the borders
    for (int64_t k = gtid; k < a.S; k += gstep) {
        a.w.tokens[k] = 0;
        a.w.bad[k] = 0;
        a.w.acc[k] = 0;
    }
    for (int64_t k = gtid; k < (int64_t)a.S * E; k += gstep) a.counts[k] = 0;
    bal_arrive(a);
    for (int64_t k = gtid; k < a.S; k += gstep) {
        const int64_t b0 = a.starts[k], b1 = a.starts[k + 1];
        if (b0 < 0 || b1 < b0 || b1 > a.T) raise_flag(a.w.status, kFlagBounds, 710);
    }

    // this block's counts, in shared memory where its tokens' sequences fit
    const int32_t* starts = a.starts;
    if (a.S < kBalStarts) {
        for (int i = tid; i <= a.S; i += kBalThreads) sh.starts[i] = a.starts[i];
        starts = sh.starts;
    }
    __syncthreads();
    if (tid == 0) sh.lo = bal_find(starts, a.S, t0);
    if (tid == 32) sh.hi = bal_find(starts, a.S, t1 - 1);
    __syncthreads();
    const int lo = sh.lo, span = sh.hi - lo + 1;
    const bool local = span >= 1 && span <= kBalSpan && (int64_t)span * E <= kBalHist;
    auto count = [&](bool in_shared) {
        for (int64_t t = t0 + tid; t < t1; t += kBalThreads) {
            int id[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) id[k] = t == t0 + tid ? first_id[k] : k < a.K ? a.ids[t * a.K + k] : 0;
            const int i = bal_sequence(a, starts, t);
            if (i < 0) continue;
            const bool here = in_shared && i >= lo && i < lo + span;
            atomicAdd(here ? &sh.tokens[i - lo] : &a.w.tokens[i], 1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k >= a.K) break;
                if (id[k] < 0 || id[k] >= E) raise_flag(a.w.status, kFlagBounds, 711);
                else if (here) atomicAdd(&sh.hist[(i - lo) * E + id[k]], 1);
                else atomicAdd(&a.counts[(int64_t)i * E + id[k]], 1);
            }
        }
    };
    // borders that do not rise can put a token outside lo .. hi: those blocks count
    // in global memory like the ones whose sequences do not fit
    bool rising = true;
    if (local) {
        for (int i = tid; i < span * E; i += kBalThreads) sh.hist[i] = 0;
        for (int i = tid; i < span; i += kBalThreads) sh.tokens[i] = 0;
        for (int i = lo + tid; i < lo + span && i < a.S; i += kBalThreads) rising &= starts[i] <= starts[i + 1];
    }
    const bool in_shared = __syncthreads_and(local && rising) != 0;
    if (in_shared) count(true);
    bal_wait(a, 1);  // the sums are zero everywhere
    if (in_shared) {
        for (int i = tid; i < span && lo + i < a.S; i += kBalThreads) {
            const int n = sh.tokens[i];
            if (n > 0) atomicAdd(&a.w.tokens[lo + i], n);
        }
        for (int i = tid; i < span * E; i += kBalThreads) {
            const int n = sh.hist[i];
            if (n > 0) atomicAdd(&a.counts[(int64_t)lo * E + i], n);
        }
    } else {
        count(false);
    }
    bal_arrive(a);

    // the tokens, kBalThreads / L at a time, the next one's logits loaded while one
    // is worked on (the first one's before the wait)
    const int lg = tid & (L - 1);
    const int64_t per = kBalThreads / L;
    float nl[kBalPer], f[kBalPer];
#pragma unroll
    for (int j = 0; j < kBalPer; ++j) nl[j] = f[j] = 0.f;
    int ni = -1, at = -1, i_of = -1;  // the next token's sequence; where it was found; the one f is of
    auto fetch = [&](int64_t t) {
        ni = -1;
        if (t >= t1) return;
        const bool on = a.mask == nullptr || a.mask[t] != 0;
        bal_load<L, VEC, float>(a.logits + t * E, lg, E, nl, -INFINITY);  // (not used where the token does not count)
        if (at < 0 || (int64_t)starts[at] > t || (int64_t)starts[at + 1] <= t) {  // most tokens stay in a sequence
            at = bal_find(starts, a.S, t);
            if (at >= a.S || (int64_t)starts[at] > t || (int64_t)starts[at + 1] <= t) at = -1;
        }
        if (on) ni = at;
    };
    fetch(t0 + tid / L);
    bal_wait(a, 2);  // the counts are complete
    // S' and N
    int my_used = 0;
    unsigned long long my_all = 0;
    for (int k = tid; k < a.S; k += kBalThreads) {
        const int n = bal_read(&a.w.tokens[k]);
        my_used += n > 0;
        my_all += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        my_used += __shfl_xor_sync(0xffffffffu, my_used, o);
        my_all += __shfl_xor_sync(0xffffffffu, my_all, o);
    }
    if ((tid & 31) == 0) {
        sh.used[tid >> 5] = my_used;
        sh.all[tid >> 5] = my_all;
    }
    __syncthreads();
    int used = 0;
    unsigned long long all = 0;
    for (int w = 0; w < kBalThreads / 32; ++w) {
        used += sh.used[w];
        all += sh.all[w];
    }
    const float cb0 = a.c_balance * (float)E / (float)used, cz0 = a.c_z * 2.f / (float)all;
    float inv_n = 0.f;
    unsigned long long acc = 0;  // of sequence i_of
    double z = 0.0;
    for (int64_t base = t0; base < t1; base += per) {
        const int64_t t = base + tid / L;
        const int i = ni;
        float l[kBalPer], p[kBalPer];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) {
            l[j] = nl[j];
            mx = fmaxf(mx, l[j]);
        }
        if (base + per < t1) fetch(t + per);
        if (L == 32 && i < 0) {  // the whole warp's token does not count, or is behind the chunk
            if (t < t1 && a.dlogits != nullptr) {
                float d[kBalPer];
#pragma unroll
                for (int j = 0; j < kBalPer; ++j) d[j] = 0.f;
                bal_store<L, VEC>(a.dlogits + t * E, lg, E, d);
            }
            continue;
        }
        if (i >= 0 && i != i_of) {
            if (acc != 0) atomicAdd(&a.w.acc[i_of], acc);
            acc = 0;
            i_of = i;
            inv_n = 1.f / (float)bal_read(&a.w.tokens[i]);
            const float fscale = inv_n / (float)a.K;
            int n[kBalPer];
            bal_load<L, VEC, int>(a.counts + (int64_t)i * E, lg, E, n, 0);
#pragma unroll
            for (int j = 0; j < kBalPer; ++j) f[j] = (float)n[j] * fscale;
        }
        // softmax: p = exp(l - max) / sum.  Sigmoid scores: l becomes score / sum of
        // scores.  Where all of a token's scores are small (largest logit m below -20) they
        // are taken in units of e^m: score e^-m = 1 / (e^m + e^(m - l)), which neither
        // underflows nor meets an infinite sum; above, m = 0 and the exponent's argument
        // is the logit itself.  1 - score is e^(m - l) times that where the score is near
        // 1, so that a saturated expert's gradient keeps its digits.
        mx = group_max<L>(mx);
        const float m = SIG && mx < -20.f ? mx : 0.f, em = SIG ? expf(m) : 1.f;
        float se = 0.f, sg = 0.f, c = 0.f, one_less[kBalPer];
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) {
            p[j] = expf(l[j] - mx);  // 0 for the lanes' places behind E, which hold -inf
            se += p[j];
            if (SIG) {
                const float t = expf(m - l[j]), sc = 1.f / (em + t);
                one_less[j] = l[j] > 0.f ? t * sc : 1.f - em * sc;
                l[j] = sc;
                sg += sc;
            }
            c = fmaf(f[j], SIG ? l[j] : p[j], c);
        }
        se = group_sum<L>(se);
        c = group_sum<L>(c);
        if (SIG) sg = group_sum<L>(sg);
        const float lse = mx + logf(se), inv_se = 1.f / se;
        const float inv_sg = SIG ? 1.f / sg : 0.f;
        c *= SIG ? inv_sg : inv_se;
        if (t >= t1) continue;
        if (i >= 0 && lg == 0) {
            z = fma((double)lse, (double)lse, z);
            if (c >= 0.f && c <= 1.5f) acc += __float2ull_rn(c * a.fix);  // (the product is exact)
            else a.w.bad[i] = 1;
        }
        if (a.dlogits != nullptr) {
            float d[kBalPer];
            const float cb = cb0 * inv_n * (SIG ? inv_sg : inv_se), cz = cz0 * lse * inv_se;
#pragma unroll
            for (int j = 0; j < kBalPer; ++j) {
                const float dp = SIG ? l[j] * one_less[j] : p[j];
                d[j] = i >= 0 ? cb * dp * (f[j] - c) + cz * p[j] : 0.f;
            }
            bal_store<L, VEC>(a.dlogits + t * E, lg, E, d);
        }
    }
    // the warp's shares of one sequence as one addition
    const int i0 = __shfl_sync(0xffffffffu, i_of, 0);
    if (__all_sync(0xffffffffu, i_of == i0 || acc == 0)) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if ((tid & 31) == 0 && acc != 0) atomicAdd(&a.w.acc[i0], acc);
    } else if (acc != 0) {
        atomicAdd(&a.w.acc[i_of], acc);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if ((tid & 31) == 0) sh.red[0][tid >> 5] = z;
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
        for (int w = 0; w < kBalThreads / 32; ++w) s += sh.red[0][w];
        a.w.zpart[blockIdx.x] = s;
        // releases this block's additions (thread 0's release covers what the block
        // barrier ordered before it) and acquires the others'
        uint32_t n;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(a.w.done) : "memory");
        sh.last = n == gridDim.x - 1;
    }
    __syncthreads();
    if (!sh.last) return;
    // the block that finishes last: per-sequence losses, then both means
    double zsum = 0.0, bsum = 0.0;
    for (int64_t b = tid; b < gridDim.x; b += kBalThreads) zsum += bal_read(&a.w.zpart[b]);
    for (int64_t k = tid; k < a.S; k += kBalThreads) {
        const int n = bal_read(&a.w.tokens[k]), bad = bal_read(&a.w.bad[k]);
        const unsigned long long sum = bal_read(&a.w.acc[k]);
        double v = 0.0;
        if (n > 0) v = bad ? (double)NAN : (double)E * (double)sum / (double)a.fix / (double)n;
        a.seq_loss[k] = (float)v;
        bsum += v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        zsum += __shfl_xor_sync(0xffffffffu, zsum, o);
        bsum += __shfl_xor_sync(0xffffffffu, bsum, o);
    }
    if ((tid & 31) == 0) {
        sh.red[0][tid >> 5] = zsum;
        sh.red[1][tid >> 5] = bsum;
    }
    __syncthreads();
    if (tid == 0) {
        *a.w.bar = 0;  // every block has passed both barriers
        *a.w.done = 0;
        double zt = 0.0, bt = 0.0;
        for (int w = 0; w < kBalThreads / 32; ++w) {
            zt += sh.red[0][w];
            bt += sh.red[1][w];
        }
        a.losses[0] = all ? (float)(zt / (double)all) : 0.f;
        a.losses[1] = used ? (float)(bt / (double)used) : 0.f;
    }
}

// ------------------------------------------------------------------- host --
struct BalLayout {
    size_t head, tokens, bad, acc, zpart, total;
};
static BalLayout balance_layout(int64_t S)
{
    BalLayout L;
    size_t o = 0;
    L.head = o;   o += 256;  // status word, then the call's counters
    L.tokens = o; o += align_up((size_t)S * 4);
    L.bad = o;    o += align_up((size_t)S * 4);
    L.acc = o;    o += align_up((size_t)S * 8);
    L.zpart = o;  o += align_up((size_t)kBalMaxBlocks * 8);
    L.total = o;
    return L;
}
size_t balance_bytes(const moe_config&, int64_t S) { return balance_layout(S).total; }

template <int L, bool VEC, bool SIG> static cudaError_t launch_balance_t(BalArgs a, cudaStream_t s)
{
    // resident blocks, per device (the launch is cooperative)
    static std::atomic<int> cached[32];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int resident = dev >= 0 && dev < 32 ? cached[dev].load(std::memory_order_acquire) : 0;
    if (resident == 0) {
        int per_sm = 0, sms = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, balance_kernel<L, VEC, SIG>, kBalThreads, 0);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        resident = per_sm * sms;
        if (resident < 1) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 32) cached[dev].store(resident, std::memory_order_release);
    }
    int64_t blocks = (a.T * L + kBalThreads - 1) / kBalThreads;
    if (blocks > resident) blocks = resident;
    if (blocks > kBalMaxBlocks) blocks = kBalMaxBlocks;
    a.chunk = (a.T + blocks - 1) / blocks;
    blocks = (a.T + a.chunk - 1) / a.chunk;  // none without tokens
    void* args[] = {&a};
    return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(balance_kernel<L, VEC, SIG>), dim3((unsigned)blocks),
                                       dim3(kBalThreads), args, 0, s);
}

template <int L> static cudaError_t launch_balance_l(const BalArgs& a, bool sigmoid, cudaStream_t s)
{
    if (sigmoid) return a.E % 4 == 0 ? launch_balance_t<L, true, true>(a, s) : launch_balance_t<L, false, true>(a, s);
    return a.E % 4 == 0 ? launch_balance_t<L, true, false>(a, s) : launch_balance_t<L, false, false>(a, s);
}

cudaError_t launch_balance(const moe_config& c, int64_t S, const float* logits, const int32_t* ids,
                           const int32_t* starts, const uint8_t* mask, float c_balance, float c_z, int32_t* counts,
                           float* losses, float* seq_loss, float* dlogits, void* ws, cudaStream_t s)
{
    const BalLayout L = balance_layout(S);
    char* w = static_cast<char*>(ws);
    BalArgs a;
    a.logits = logits; a.ids = ids; a.starts = starts; a.mask = mask;
    a.counts = counts; a.losses = losses; a.seq_loss = seq_loss; a.dlogits = dlogits;
    a.T = c.T; a.chunk = 0; a.E = c.E; a.K = c.K; a.S = (int)S;
    const bool sigmoid = c.score_func == MOE_SCORE_SIGMOID;
    a.c_balance = c_balance; a.c_z = c_z;
    int bits = 0;
    while (c.T >> bits != 0) ++bits;
    a.fix = ldexpf(1.f, 63 - bits);
    a.w.status = reinterpret_cast<int*>(w + L.head);
    a.w.bar = reinterpret_cast<uint32_t*>(w + L.head + 64);
    a.w.done = reinterpret_cast<uint32_t*>(w + L.head + 128);
    a.w.tokens = reinterpret_cast<int*>(w + L.tokens);
    a.w.bad = reinterpret_cast<int*>(w + L.bad);
    a.w.acc = reinterpret_cast<unsigned long long*>(w + L.acc);
    a.w.zpart = reinterpret_cast<double*>(w + L.zpart);
    if (c.E <= 8) return launch_balance_l<1>(a, sigmoid, s);
    if (c.E <= 16) return launch_balance_l<2>(a, sigmoid, s);
    if (c.E <= 32) return launch_balance_l<4>(a, sigmoid, s);
    if (c.E <= 64) return launch_balance_l<8>(a, sigmoid, s);
    if (c.E <= 128) return launch_balance_l<16>(a, sigmoid, s);
    return launch_balance_l<32>(a, sigmoid, s);
}

}  // namespace moe
