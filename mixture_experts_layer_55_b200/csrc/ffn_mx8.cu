// ffn_mx8.cu -- grouped SwiGLU experts on 8-bit rows and weights, on the tensor
// cores' block-scaled MMA (tcgen05, kind::mxf8f6f4).
//
// Rows and weights are e4m3 in blocks of 32 along the contracted axis with
// power-of-two scales (mx8.cuh); for every row r of expert e
//   g = x_r . Wg_e,  u = x_r . Wu_e                       (K = D, fp32 sums)
//   h_r = 8-bit blocks of silu(g) u                       (blocks of 32 along F)
//   y_r = bf16(w_r (h_r . Wd_e))                          (K = F)
// h is rounded to 8 bits straight from the fp32 accumulators: at most 2^-4 of a
// value, the precision of every operand of these products.
//
// Persistent kernel on the tiles of the bf16 experts (ffn_tc.cu): 128 rows per
// CTA, or 256 per CTA pair (cta_group::2), by 256 accumulator columns (gate/up:
// 128 of F, gate and up interleaved in blocks of 64; down: 256 of D).  A stage
// is 128 of the contracted axis: one 128-byte swizzle row of A and of B (both
// K-major), four MMAs of K = 32, each with one scale per row.  14 warps per CTA:
//   warp 0       TMA producer: A 128 x 128 and B 256 (pair: 128) x 128 bytes
//   warp 1       MMA issuer (pair: the leader's); owns the tensor memory
//   warps 2..5   scales: a thread per row of A and two of B loads the scales of
//                four stages at once (16 bytes of a row where rows allow it), two
//                such groups ahead, and writes each stage's as 32 x 16-byte blocks
//                [row % 32][row / 32][4 of K] into a ring of four groups;
//                tcgen05.cp replicates them over the four lane quadrants of
//                tensor memory
//   warps 6..13  epilogue: two per lane quadrant, each half of the columns
// Tensor memory: two accumulators of 256 columns and the scales do not fit 512
// columns, so the accumulators overlap by 32 (0..255 and 224..479, scales from
// 480).  The epilogue empties the shared columns first and says so; the next
// tile's MMAs start then, not when the whole accumulator has been read.
//
// Bound: the tensor cores, under the power cap.  Measured on the way (T = 4096,
// D = F = 4096, 8 experts, K = 2; gate/up and down in us): 461 + 232 with a
// release at cluster scope for every stage's scales; 351 + 182 with one for every
// four stages, issued by an idle thread; 276 + 141 with the issuing warp's
// operands in uniform registers; 232 + 126 with scales four groups deep and
// 32-byte stores.  The MMAs alone take 184 + 97, the loads alone 165 + 84.
// T = 8192, D = 4096, F = 14336: 2.25 ms for single calls (2570 TFLOP/s), 2.6-2.7 ms
// back to back at the 1000 W cap (1.33 GHz).
#include <cuda.h>

#include "internal.h"
#include "mx8.cuh"

namespace moe {

// ffn_tc.cu: the per-expert A maps (row extent cut to the expert's end)
cudaError_t launch_ffn_amaps(const void* map_x, const void* map_h, const int32_t* offsets, int E, int64_t max_rows,
                             void* maps, cudaStream_t s);

namespace mx {

constexpr int BK = 128;                // contracted elements (bytes) per stage
constexpr int A_BYTES = 128 * BK;
constexpr int SF_BYTES = 3 * 512;      // a stage's scales: 128 rows of A and 256 of B, 4 per row
constexpr int SF_GROUP = 4;            // stages whose scales arrive together (1, 2 or 4)
constexpr int SF_SLOTS = 16 / SF_GROUP;  // groups in shared memory
constexpr int SF_SLOT_BYTES = SF_GROUP * SF_BYTES;
constexpr int ACC_STRIDE = 224;        // second accumulator's first column
constexpr int SF_COL = 480;            // scales: two buffers, A's 4 columns, then B's 8
constexpr int SF_BUF_COLS = 16;
constexpr int TMEM_COLS = 512;
constexpr int SF_WARPS = 4;
constexpr int EPI_WARPS = 8;
constexpr int EPI_WARP0 = 2 + SF_WARPS;
constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int MAX_E = 256;
// Average rows per expert up to which tokens are the MMA's columns.  Measured on
// balanced loads (8 experts, D = 4096, F = 14336; as columns and as rows): 16 rows 227 and 244 us,
// 32 rows 271 and 244; 64 experts, D = 2048, F = 1408: 6 rows 97 and 100, 24 rows
// 101 and 105, 32 rows 105 and 104, 48 rows 121 and 106.
constexpr int kFewRows = 24;

template <bool GATEUP, bool PAIR> struct Geo {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int BM = 128 * CTAS;
    static constexpr int B_ROWS = 256 / CTAS;              // rows of B in this CTA
    static constexpr int B_BYTES = B_ROWS * BK;
    static constexpr int OP_BYTES = A_BYTES + B_BYTES;     // one stage's operands
    // a pair's down product gives one operand stage for 64-column pieces of y, 4 KB
    // per epilogue warp, that leave by TMA in whole lines
    static constexpr bool STAGED = PAIR && !GATEUP;
    static constexpr int OUT_BYTES = STAGED ? 4096 : 0;
    static constexpr int STAGES = STAGED ? 5 : PAIR ? 6 : 4;
};

struct Misc {
    uint64_t full[8];
    uint64_t empty[8];
    uint64_t sfull[SF_SLOTS];   // a group's scales are in shared memory (both CTAs')
    uint64_t sempty[SF_SLOTS];  // and have been copied to tensor memory
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t tover;       // the accumulators' shared columns have been read
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int row0[MAX_E];
    int rowend[MAX_E];
    int pref[MAX_E + 1];
    int warp_sum[NUM_THREADS / 32];
};

template <bool GATEUP, bool PAIR> constexpr size_t smem_bytes()
{
    using G = Geo<GATEUP, PAIR>;
    return 1024 + (size_t)G::STAGES * G::OP_BYTES + EPI_WARPS * G::OUT_BYTES + SF_SLOTS * SF_SLOT_BYTES + sizeof(Misc);
}

struct Args {
    const int32_t* offsets;
    const int32_t* perm;
    const float* topk_w;
    const uint8_t* as;         // A's scales (rows, Kdim / 32)
    const uint8_t *b0s, *b1s;  // B's scales (E, N, Kdim / 32): gate or down; up
    uint8_t *h, *hs;           // gate/up's output
    __nv_bfloat16* y;          // down's
    int E, Kdim, N, n_tiles;
    int64_t max_rows, nk;
    int* status;
    const CUtensorMap* amaps;  // A's map per expert (null: tmA)
    int splits;                // few rows, down: the contracted axis is cut in this many parts
    float* part;               // their sums (splits, max_rows, N) where splits > 1
};

// ------------------------------------------------------------------- PTX --
// Instruction descriptor of kind::mxf8f6f4: e4m3 operands (format 0), scales of
// type UE8M0 (bit 23); bits 4-5 and 29-30 pick the scale byte of B and of A.
MOE_DEVICE constexpr uint32_t mx_idesc(int M, int N)
{
    return (1u << 23) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The issuing warp runs as a whole (its operands stay in uniform registers) and
// one elected lane (`leader`) issues: with a single-lane branch around the loop
// instead, moving the operands took 80 cycles for each MMA, more than half of
// the MMA itself, and bound the kernel.
template <bool PAIR>
MOE_DEVICE void mma_mx8(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                        uint32_t sfb, uint32_t accumulate)
{
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(leader)
            : "memory");
}

// 32 x 16 bytes of shared memory to four columns, replicated over the lane
// quadrants (pair: in both CTAs, each from its own shared memory).
template <bool PAIR> MOE_DEVICE void copy_scales(uint32_t leader, uint32_t taddr, uint64_t desc)
{
    if (PAIR)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(desc), "r"(leader)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(desc), "r"(leader)
                     : "memory");
}

// Arrive on the barrier (pair: at this offset in both CTAs) once every tensor
// instruction that the elected lane has issued so far is done.
template <bool PAIR> MOE_DEVICE void commit(uint32_t leader, uint32_t bar)
{
    if (PAIR)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
                     "h"((uint16_t)0x3), "r"(leader)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                     "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
                     "r"(leader)
                     : "memory");
}

// Descriptor of a block of scales: no swizzle, groups of 8 rows 128 bytes apart.
MOE_DEVICE uint64_t scale_desc(uint32_t smem_addr)
{
    return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1u << 46);
}

// All lanes wait, and agree on the outcome.
MOE_DEVICE bool warp_wait_all(uint64_t* bar, uint32_t parity, int* status, int where, volatile int* abort_flag)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, where, abort_flag));
}

// One lane waits for the warp.
MOE_DEVICE bool warp_wait(uint64_t* bar, uint32_t parity, int lane, int* status, int where, volatile int* abort_flag)
{
    int ok = 1;
    if (lane == 0) ok = mbar_wait(bar, parity, status, where, abort_flag) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Arrival on the leader's barrier that says tensor memory has been read (the
// loads are complete: tcgen05.wait::ld).  No memory is published with it, so it
// needs no release at cluster scope, which costs about 1000 cycles here.
MOE_DEVICE void arrive_read(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// ----------------------------------------------------------------- tiles --
MOE_DEVICE void decode_tile(const Misc* m, int E, int bm, int bn, int t, int& e, int& m_row0, int& row_end, int& n0)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {  // largest e with pref[e] <= t (its block is non-empty)
        const int mid = (lo + hi + 1) >> 1;
        if (m->pref[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    e = lo;
    const int mt = (m->rowend[e] - m->row0[e] + bm - 1) / bm;
    const int local = t - m->pref[e];
    const int n = local / mt, mm = local - n * mt;
    m_row0 = m->row0[e] + mm * bm;
    row_end = m->rowend[e];
    n0 = n * bn;
}

// The tile table from the offsets, a thread per expert (with offsets that are
// malformed anywhere nothing is computed).  Every thread of the block calls it.
MOE_DEVICE void build_tiles(Misc* m, const Args& a, int bm)
{
    const int e = threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int tiles = 0;
    bool bad = false;
    if (e < a.E) {
        const int r0 = a.offsets[e], r1 = a.offsets[e + 1];
        bad = r0 < 0 || r1 < r0 || (int64_t)r1 > a.max_rows;
        m->row0[e] = r0;
        m->rowend[e] = r1;
        if (!bad) tiles = (r1 - r0 + bm - 1) / bm * a.n_tiles;
    }
    const bool any_bad = __syncthreads_or(bad) != 0;
    if (any_bad && threadIdx.x == 0) raise_flag(a.status, kFlagBounds, 720);
    if (any_bad) tiles = 0;
    int run = tiles;  // inclusive sum within the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
    }
    if (lane == 31) m->warp_sum[warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; ++w) run += m->warp_sum[w];
    if (e < a.E) m->pref[e + 1] = run;
    if (e == 0) m->pref[0] = 0;
}

// Scales of stages 4g .. 4g+3 of one row (null: zeros), nb = bytes per row.
// Rows are 16-byte, 4-byte or only byte aligned with nb.  WEIGHT: of a weight, which
// nothing writes while the kernel runs (the read-only path).  The rows' scales of the
// down product are written by the gate/up product while this kernel is already
// resident: ordinary loads, which the wait for that product orders.
template <bool WEIGHT, typename V> MOE_DEVICE V load_scale(const uint8_t* p)
{
    return WEIGHT ? __ldg(reinterpret_cast<const V*>(p)) : *reinterpret_cast<const V*>(p);
}
template <bool WEIGHT> MOE_DEVICE uint4 load_scales(const uint8_t* row, int g, int nb)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row == nullptr) return v;
    if ((nb & 15) == 0) return load_scale<WEIGHT, uint4>(row + 16 * g);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 16 * g + 4 * i;
        w[i] = 0;
        if ((nb & 3) == 0) {
            if (at < nb) w[i] = load_scale<WEIGHT, uint32_t>(row + at);
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (at + b < nb) w[i] |= (uint32_t)load_scale<WEIGHT, uint8_t>(row + at + b) << (8 * b);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

MOE_DEVICE uint32_t word_of(const uint4& v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// 32 bytes at a 32-byte boundary in one store: a whole sector per lane.
MOE_DEVICE void store32(void* p, const uint32_t* v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// silu(g) u in fp32: g u / (1 + e^-g) for g >= 0, g e^g u / (1 + e^g) below, so that the
// divisor stays in 1 .. 2 (from e^87 on the fast quotient gives 0, and a large u would
// have shown it).  The exponential errs by 2 + 1.2 |g| units of 2^-23 at most, the quotient
// by 2: 2^-20 of the value up to |g| = 3, 2^-18 up to 20; h is then rounded to 2^-4.
MOE_DEVICE float swiglu(float g, float u)
{
    const float e = __expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * e : g, 1.0f + e) * u;
}

template <bool GATEUP, bool PAIR>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    ffn_mx8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                   const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmY, const Args a)
{
    using G = Geo<GATEUP, PAIR>;
    constexpr int BM = G::BM, BN = GATEUP ? 128 : 256, STAGES = G::STAGES, OP_BYTES = G::OP_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stages = smem;
    uint8_t* outbuf = smem + (size_t)STAGES * OP_BYTES;  // EPI_WARPS x OUT_BYTES, 1 KB aligned
    uint8_t* scales = outbuf + (size_t)EPI_WARPS * G::OUT_BYTES;
    Misc* m = reinterpret_cast<Misc*>(scales + (size_t)SF_SLOTS * SF_SLOT_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;  // 0: the leader, which issues the MMAs
    const int unit = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int units = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&m->full[s], 1);
            mbar_init(&m->empty[s], 1);
        }
        for (int s = 0; s < SF_SLOTS; ++s) {
            mbar_init(&m->sfull[s], SF_WARPS + (PAIR && rank == 0 ? 1 : 0));  // leader: and the peer's
            mbar_init(&m->sempty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&m->tfull[b], 1);
            mbar_init(&m->tempty[b], EPI_WARPS * G::CTAS);
        }
        mbar_init(&m->tover, EPI_WARPS / 2 * G::CTAS);
        mbar_init(&m->drain, 1);
        m->abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB0);
        if (GATEUP) prefetch_tmap(&tmB1);
        if (G::STAGED) prefetch_tmap(&tmY);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(&m->tmem_base, TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&m->tmem_base, TMEM_COLS);
            tmem_relinquish();
        }
    }
    build_tiles(m, a, BM);
    tc_fence_before();
    if (PAIR) cluster_sync();  // the peer's barriers are initialised before any remote signal
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = m->tmem_base;
    const int total = m->pref[E];
    const int num_kb = (a.Kdim + BK - 1) / BK;
    volatile int* abort_flag = &m->abort_flag;

    // The down product is launched while the gate/up product still runs: what reads
    // h waits until that has ended, the rest of its start does not.
    if (GATEUP) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer (each CTA)
            if (!GATEUP) asm volatile("griddepcontrol.wait;" ::: "memory");
            int stage = 0;
            uint32_t phase = 0;
            int last_phase[STAGES];
            for (int s = 0; s < STAGES; ++s) last_phase[s] = -1;
            bool ok = true;
            int last_e = -1;
            for (int t = unit; t < total && ok; t += units) {
                int e, m_row0, row_end, n0;
                decode_tile(m, E, BM, BN, t, e, m_row0, row_end, n0);
                const int a_row = m_row0 + (int)rank * 128;
                const CUtensorMap* mA = &tmA;
                if (a.amaps != nullptr) {  // the expert's own map: rows past its end read as zeros
                    mA = a.amaps + e;
                    if (e != last_e) {
                        asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(mA) : "memory");
                        last_e = e;
                    }
                }
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&m->empty[stage], phase ^ 1u, a.status, 722, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sA = stages + (size_t)stage * OP_BYTES;
                    uint8_t* sB = sA + A_BYTES;
                    const int k0 = kb * BK;
                    if (PAIR) {
                        // both CTAs' bytes are counted on the leader's barrier
                        if (rank == 0) mbar_arrive_expect_tx(&m->full[stage], 2 * OP_BYTES);
                        const uint32_t fb = mapa_shared(smem_u32(&m->full[stage]), 0);
                        tma_load_2d_pair(sA, mA, k0, a_row, fb);
                        if (GATEUP) {  // this CTA's [gate 64 | up 64]
                            tma_load_3d_pair(sB, &tmB0, k0, n0 + 64 * (int)rank, e, fb);
                            tma_load_3d_pair(sB + 64 * BK, &tmB1, k0, n0 + 64 * (int)rank, e, fb);
                        } else {
                            tma_load_3d_pair(sB, &tmB0, k0, n0 + 128 * (int)rank, e, fb);
                            tma_load_3d_pair(sB + 64 * BK, &tmB0, k0, n0 + 128 * (int)rank + 64, e, fb);
                        }
                    } else {
                        uint64_t* fb = &m->full[stage];
                        mbar_arrive_expect_tx(fb, OP_BYTES);
                        tma_load_2d(sA, mA, k0, a_row, fb);
                        if (GATEUP) {  // [gate | up | gate | up], 64 each
                            tma_load_3d(sB, &tmB0, k0, n0, e, fb);
                            tma_load_3d(sB + 64 * BK, &tmB1, k0, n0, e, fb);
                            tma_load_3d(sB + 128 * BK, &tmB0, k0, n0 + 64, e, fb);
                            tma_load_3d(sB + 192 * BK, &tmB1, k0, n0 + 64, e, fb);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tma_load_3d(sB + 64 * j * BK, &tmB0, k0, n0 + 64 * j, e, fb);
                        }
                    }
                    last_phase[stage] = (int)phase;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // never leave the CTA with a copy in flight (the leader sees every completion)
            if (!PAIR || rank == 0)
                for (int s = 0; s < STAGES; ++s)
                    if (last_phase[s] >= 0) mbar_wait(&m->full[s], (uint32_t)last_phase[s], a.status, 723, nullptr);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------------------------ MMA issuer (leader CTA only)
            constexpr uint32_t idesc = mx_idesc(BM, 256);
            const uint32_t leader = elect_one();
            const uint32_t tbase = __shfl_sync(0xffffffffu, tmem_base, 0);
            const int tiles = __shfl_sync(0xffffffffu, total, 0);
            const uint32_t s_stages = __shfl_sync(0xffffffffu, smem_u32(stages), 0);
            const uint32_t s_scales = __shfl_sync(0xffffffffu, smem_u32(scales), 0);
            const uint32_t s_empty = __shfl_sync(0xffffffffu, smem_u32(&m->empty[0]), 0);
            const uint32_t s_sempty = __shfl_sync(0xffffffffu, smem_u32(&m->sempty[0]), 0);
            const uint32_t s_tfull = __shfl_sync(0xffffffffu, smem_u32(&m->tfull[0]), 0);
            int stage = 0, acc = 0, slot = 0, in_slot = 0;
            uint32_t phase = 0, acc_phase = 0, sphase = 0, over_phase = 1;  // no tile before the first one
            bool ok = true;
            for (int t = unit; t < tiles && ok; t += units) {
                // this accumulator's last tile has been read, and the shared
                // columns of the tile before this one
                if (!warp_wait_all(&m->tempty[acc], acc_phase ^ 1u, a.status, 724, abort_flag)) break;
                if (!warp_wait_all(&m->tover, over_phase, a.status, 725, abort_flag)) break;
                over_phase ^= 1u;
                tc_fence_after();
                const uint32_t d0 = tbase + (uint32_t)(acc * ACC_STRIDE);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (in_slot == 0 && !warp_wait_all(&m->sfull[slot], sphase, a.status, 727, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (!warp_wait_all(&m->full[stage], phase, a.status, 726, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // the copies and the MMAs of one thread run in order
                    const uint32_t tsa = tbase + SF_COL + (uint32_t)((kb & 1) * SF_BUF_COLS);
                    const uint64_t sdesc = scale_desc(s_scales + (uint32_t)(slot * SF_SLOT_BYTES + in_slot * SF_BYTES));
                    copy_scales<PAIR>(leader, tsa, sdesc);
                    copy_scales<PAIR>(leader, tsa + 4, sdesc + (512 >> 4));
                    copy_scales<PAIR>(leader, tsa + 8, sdesc + (1024 >> 4));
                    const uint64_t adesc = umma_desc_sw128(s_stages + (uint32_t)stage * OP_BYTES, 16, 1024);
                    const uint64_t bdesc = adesc + (A_BYTES >> 4);
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        mma_mx8<PAIR>(leader, d0, adesc + kk * 2, bdesc + kk * 2,
                                      idesc | ((uint32_t)kk << 4) | ((uint32_t)kk << 29), tsa, tsa + 4,
                                      kk != 0 ? 1u : (kb != 0 ? 1u : 0u));
                    // frees the stage (in both CTAs) once these complete
                    commit<PAIR>(leader, s_empty + (uint32_t)stage * 8);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++in_slot == SF_GROUP || kb == num_kb - 1) {  // and the group's scales
                        commit<PAIR>(leader, s_sempty + (uint32_t)slot * 8);
                        in_slot = 0;
                        if (++slot == SF_SLOTS) {
                            slot = 0;
                            sphase ^= 1u;
                        }
                    }
                }
                if (!ok) break;
                commit<PAIR>(leader, s_tfull + (uint32_t)acc * 8);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            // every MMA issued here is done before the allocation is released
            __syncwarp();
            if (leader) {
                if (PAIR) umma_commit_pair_mc(&m->drain, 0x1);
                else umma_commit(&m->drain);
            }
            __syncwarp();
            warp_wait_all(&m->drain, 0, a.status, 728, nullptr);
        } else if (PAIR && lane == 0) {
            // ------------------------------------------------ the peer: its scales' arrival, passed on
            // The release at cluster scope that makes them the leader's to use
            // waits for the issuing thread's own memory traffic, about 1000 cycles
            // in a thread that loads scales; this one has none.
            int slot = 0;
            uint32_t sphase = 0;
            const int64_t mine = unit < total ? (int64_t)((total - unit + units - 1) / units) * ((num_kb + SF_GROUP - 1) / SF_GROUP) : 0;
            for (int64_t n = 0; n < mine; ++n) {
                if (!mbar_wait(&m->sfull[slot], sphase, a.status, 731, abort_flag)) break;
                mbar_arrive_cluster(mapa_shared(smem_u32(&m->sfull[slot]), 0));
                if (++slot == SF_SLOTS) {
                    slot = 0;
                    sphase ^= 1u;
                }
            }
        }
    } else if (warp < EPI_WARP0) {
        // ------------------------------------------------ scales (each CTA: its A rows, all of B's)
        if (!GATEUP) asm volatile("griddepcontrol.wait;" ::: "memory");
        const int i = (warp - 2) * 32 + lane;
        const int nb = a.Kdim / kMxBlock, groups = (num_kb + 3) / 4;
        const uint32_t off = (uint32_t)((i & 31) * 16 + (i >> 5) * 4);
        const uint8_t *pa = nullptr, *pb0 = nullptr, *pb1 = nullptr;
        auto rows_of = [&](int t) {
            int e, m_row0, row_end, n0;
            decode_tile(m, E, BM, BN, t, e, m_row0, row_end, n0);
            const int64_t row = (int64_t)m_row0 + (int)rank * 128 + i;
            pa = row < row_end ? a.as + row * nb : nullptr;
            // accumulator columns i and 128 + i: gate/up blocks of 64, or down
            const uint8_t* bs = GATEUP && i >= 64 ? a.b1s : a.b0s;
            const int n = GATEUP ? n0 + (i & 63) : n0 + i;
            const int n2 = GATEUP ? n + 64 : n + 128;
            const int64_t be = (int64_t)e * a.N;
            pb0 = n < a.N ? bs + (be + n) * nb : nullptr;
            pb1 = n2 < a.N ? bs + (be + n2) * nb : nullptr;
        };
        // two groups of loads in flight; a group's are long done when the fence of
        // the one before it, which waits for loads too, is reached
        uint4 va[2], v0[2], v1[2];
        int ld_t = unit, ld_g = 0;
        auto load_next = [&](int i2) {
            if (ld_t >= total) return;
            if (ld_g == 0) rows_of(ld_t);
            va[i2] = load_scales<false>(pa, ld_g, nb);
            v0[i2] = load_scales<true>(pb0, ld_g, nb);
            v1[i2] = load_scales<true>(pb1, ld_g, nb);
            if (++ld_g == groups) {
                ld_g = 0;
                ld_t += units;
            }
        };
        load_next(0);
        load_next(1);
        int slot = 0, kb_left = num_kb;
        uint32_t sphase = 0;
        const int64_t mine = unit < total ? (int64_t)((total - unit + units - 1) / units) * groups : 0;
        for (int64_t n = 0; n < mine; n += 2) {
            bool ok = true;
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
                if (n + i2 >= mine) break;
#pragma unroll
                for (int h = 0; h < 4 / SF_GROUP; ++h) {
                    if (kb_left <= h * SF_GROUP) break;  // the tile's last stages
                    if (!warp_wait(&m->sempty[slot], sphase ^ 1u, lane, a.status, 729, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t* dst = scales + (size_t)slot * SF_SLOT_BYTES + off;
#pragma unroll
                    for (int k = 0; k < SF_GROUP; ++k) {
                        *reinterpret_cast<uint32_t*>(dst + k * SF_BYTES) = word_of(va[i2], h * SF_GROUP + k);
                        *reinterpret_cast<uint32_t*>(dst + k * SF_BYTES + 512) = word_of(v0[i2], h * SF_GROUP + k);
                        *reinterpret_cast<uint32_t*>(dst + k * SF_BYTES + 1024) = word_of(v1[i2], h * SF_GROUP + k);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m->sfull[slot]);
                    if (++slot == SF_SLOTS) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                }
                if (!ok) break;
                kb_left -= 4;
                if (kb_left <= 0) kb_left = num_kb;
                load_next(i2);
            }
            if (!ok) break;
        }
    } else {
        // ------------------------------------------------ epilogue (each CTA, its 128 rows)
        const int quad = warp & 3;
        const int half = (warp - EPI_WARP0) >> 2;
        const int r_in_tile = (int)rank * 128 + quad * 32 + lane;
        const uint32_t tempty0 = mapa_shared(smem_u32(&m->tempty[0]), 0);
        const uint32_t tempty1 = mapa_shared(smem_u32(&m->tempty[1]), 0);
        const uint32_t tover = mapa_shared(smem_u32(&m->tover), 0);
        uint8_t* obuf = outbuf + (size_t)(warp - EPI_WARP0) * G::OUT_BYTES;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int t = unit; t < total; t += units) {
            int e, m_row0, row_end, n0;
            decode_tile(m, E, BM, BN, t, e, m_row0, row_end, n0);
            const int64_t row = (int64_t)m_row0 + r_in_tile;
            const bool valid = row < row_end;
            float w = 1.f;  // the row's weight, loaded while the tile is computed
            if (!GATEUP && valid && a.perm != nullptr) {
                const int32_t pa = a.perm[row];
                w = 0.f;
                if (pa >= 0 && (int64_t)pa < a.nk) w = a.topk_w[pa];
                else if (half == 0) raise_flag(a.status, kFlagBounds, 721);
            }
            if (!warp_wait(&m->tfull[acc], acc_phase, lane, a.status, 730, abort_flag)) break;
            tc_fence_after();
            // the warp's 32 rows all belong to the expert: its pieces leave by TMA
            const int64_t warp_row0 = (int64_t)m_row0 + (int)rank * 128 + quad * 32;
            const bool staged = G::STAGED && warp_row0 + 32 <= row_end;
            const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * ACC_STRIDE);
            // the shared columns: the last 32 of accumulator 0, the first 32 of 1
            const bool shared_half = half == (acc == 0 ? 1 : 0);
            constexpr int CHUNKS = GATEUP ? 2 : 4;
#pragma unroll 1
            for (int cc = 0; cc < CHUNKS; ++cc) {
                const int c = half * CHUNKS + (acc == 0 ? CHUNKS - 1 - cc : cc);
                const int col = n0 + c * 32;
                uint32_t v[32], u[32];
                if (GATEUP) {  // columns [gate 0-63 | up 0-63 | gate 64-127 | up 64-127]
                    const uint32_t gcol = (uint32_t)((c >> 1) * 128 + (c & 1) * 32);
                    tmem_ld_32x32b_x32(taddr + gcol, v);
                    tmem_ld_32x32b_x32(taddr + gcol + 64, u);
                } else {
                    tmem_ld_32x32b_x32(taddr + c * 32, v);
                }
                tmem_ld_wait();
                if (cc == 0 && shared_half) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR) arrive_read(tover);
                        else mbar_arrive(&m->tover);
                    }
                }
                if (staged && (cc & 1) == 0) {  // the last piece has been read
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
                }
                if (GATEUP) {
                    if (valid && col < a.N) {
                        uint32_t mx = 0;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float h = swiglu(__uint_as_float(v[j]), __uint_as_float(u[j]));
                            v[j] = __float_as_uint(h);
                            mx = max(mx, abs_bits(h));
                        }
                        const uint32_t b = mx_scale_byte(mx);
                        const float inv = mx_inv_scale(b);
                        uint32_t p[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            p[j] = mx_pack4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                            __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]), inv);
                        store32(a.h + row * a.N + col, p);
                        a.hs[row * (a.N / kMxBlock) + col / kMxBlock] = (uint8_t)b;
                    }
                } else if (col < a.N) {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        p[j] = pack_bf16x2(w * __uint_as_float(v[2 * j]), w * __uint_as_float(v[2 * j + 1]));
                    if (!staged) {
                        if (valid) {
                            store32(a.y + row * a.N + col, p);
                            store32(a.y + row * a.N + col + 16, p + 8);
                        }
                    } else {
                        // half a row of the piece (128-byte swizzle: 16-byte part q of row r at
                        // part q ^ (r & 7))
                        uint4* dst = reinterpret_cast<uint4*>(obuf + lane * 128);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            dst[((c & 1) * 4 + q) ^ (lane & 7)] =
                                make_uint4(p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]);
                    }
                }
                if (staged && (cc & 1) == 1 && (col & ~63) < a.N) {  // columns past N fall outside the map
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tmY, obuf, col & ~63, (int)warp_row0);
                        bulk_commit();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) arrive_read(acc == 0 ? tempty0 : tempty1);
                else mbar_arrive(&m->tempty[acc]);
            }
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (G::STAGED) {
            if (lane == 0) bulk_wait_all<0>();  // every store of this warp has completed
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncwarp();
    if (PAIR) cluster_sync();  // no CTA leaves while its peer may still signal it
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------- few rows per expert --
// The same products with the operands' places exchanged: 128 rows of a weight are
// the MMA's rows and up to NT tokens its columns, so a tile of few tokens costs NT
// columns of multiplications instead of 128 padded rows.  (The weight stream is
// the bound either way, but the padded form draws the card's whole power, and at
// 880 MHz falls behind the stream: 128 tokens on 256 experts, D = 7168, F = 2048,
// 1.95 ms, against 1.68 here, 6.9 TB/s.)  A tile is two
// blocks of 128 weight rows, gate and up of the same 128 of F, or 256 of D, each
// with an accumulator of NT columns; accumulators and scales are double-buffered in
// tensor memory side by side.  In the epilogue a lane is a weight row: 32 lanes
// hold one token's block of 32 along F, whose maximum is one warp reduction.
template <int NT> struct Few {
    static constexpr int W_BYTES = 128 * BK;
    static constexpr int T_BYTES = NT * BK;
    static constexpr int OP_BYTES = 2 * W_BYTES + T_BYTES;
    static constexpr int STAGES = 5;
    static constexpr int SF_COL = 4 * NT;  // behind 2 x 2 accumulators; then A0, A1, B: 4 columns each
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * OP_BYTES + SF_SLOTS * SF_SLOT_BYTES + sizeof(Misc);
    static constexpr int TMEM = NT == 32 ? 256 : 128;
    static_assert(SF_COL + 2 * SF_BUF_COLS <= TMEM, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int N> MOE_DEVICE void tmem_ld(uint32_t taddr, uint32_t (&r)[N]);
template <> MOE_DEVICE void tmem_ld<32>(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_32x32b_x32(taddr, r); }
template <> MOE_DEVICE void tmem_ld<16>(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
template <> MOE_DEVICE void tmem_ld<8>(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

template <bool GATEUP, int NT, bool CUT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    ffn_mx8_few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW0,
                       const __grid_constant__ CUtensorMap tmW1, const Args a)
{
    using G = Few<NT>;
    constexpr int BN = GATEUP ? 128 : 256, STAGES = G::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* scales = stages + (size_t)STAGES * G::OP_BYTES;
    Misc* m = reinterpret_cast<Misc*>(scales + (size_t)SF_SLOTS * SF_SLOT_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = a.E, unit = (int)blockIdx.x, units = (int)gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&m->full[s], 1);
            mbar_init(&m->empty[s], 1);
        }
        for (int s = 0; s < SF_SLOTS; ++s) {
            mbar_init(&m->sfull[s], SF_WARPS);
            mbar_init(&m->sempty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&m->tfull[b], 1);
            mbar_init(&m->tempty[b], EPI_WARPS);
        }
        mbar_init(&m->drain, 1);
        m->abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmW0);
        if (GATEUP) prefetch_tmap(&tmW1);
    }
    if (warp == 1) {
        tmem_alloc(&m->tmem_base, G::TMEM);
        tmem_relinquish();
    }
    build_tiles(m, a, NT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = m->tmem_base;
    const int splits = CUT ? a.splits : 1;
    const int total = m->pref[E] * splits;  // work items: (tile, part of the contracted axis)
    const int num_kb = (a.Kdim + BK - 1) / BK, groups = (num_kb + 3) / 4;
    // an item's stages are whole groups of four, so that its scales' loads stay aligned
    auto first_group = [&](int sp) { return groups * sp / splits; };
    auto end_kb = [&](int sp) { return sp == splits - 1 ? num_kb : 4 * first_group(sp + 1); };
    volatile int* abort_flag = &m->abort_flag;
    // the down product starts under the gate/up product's end, as above
    if (GATEUP) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            auto weights = [&](int stage, int kb, int e, int n0) {
                uint8_t* sW = stages + (size_t)stage * G::OP_BYTES;
                mbar_arrive_expect_tx(&m->full[stage], G::OP_BYTES);
                tma_load_3d(sW, &tmW0, kb * BK, n0, e, &m->full[stage]);
                tma_load_3d(sW + G::W_BYTES, GATEUP ? &tmW1 : &tmW0, kb * BK, GATEUP ? n0 : n0 + 128, e,
                            &m->full[stage]);
            };
            auto tokens = [&](int stage, int kb, int m_row0) {
                tma_load_2d(stages + (size_t)stage * G::OP_BYTES + 2 * G::W_BYTES, &tmX, kb * BK, m_row0,
                            &m->full[stage]);
            };
            int stage = 0;
            uint32_t phase = 0;
            int last_phase[STAGES];
            for (int s = 0; s < STAGES; ++s) last_phase[s] = -1;
            bool ok = true;
            // down: the first stages' weights do not wait for h
            int early = 0;
            if (!GATEUP) {
                if (unit < total) {
                    int e, m_row0, row_end, n0;
                    decode_tile(m, E, NT, BN, unit / splits, e, m_row0, row_end, n0);
                    const int kb0 = 4 * first_group(unit % splits), n = end_kb(unit % splits) - kb0;
                    early = n < STAGES ? n : STAGES;
                    for (int st = 0; st < early; ++st) weights(st, kb0 + st, e, n0);
                }
                asm volatile("griddepcontrol.wait;" ::: "memory");
            }
            for (int t = unit; t < total && ok; t += units) {
                int e, m_row0, row_end, n0;
                decode_tile(m, E, NT, BN, t / splits, e, m_row0, row_end, n0);
                const int kb1 = end_kb(t % splits);
                for (int kb = 4 * first_group(t % splits); kb < kb1; ++kb) {
                    if (!mbar_wait(&m->empty[stage], phase ^ 1u, a.status, 742, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (early > 0) --early;
                    else weights(stage, kb, e, n0);
                    tokens(stage, kb, m_row0);
                    last_phase[stage] = (int)phase;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // never leave the CTA with a copy in flight (after an abort: stages whose
            // weights came early get their tokens too, so that their phase completes)
            for (int s = 0; early > 0 && s < STAGES; ++s)
                if (last_phase[s] < 0) {
                    tokens(s, 0, 0);
                    last_phase[s] = 0;
                    --early;
                }
            for (int s = 0; s < STAGES; ++s)
                if (last_phase[s] >= 0) mbar_wait(&m->full[s], (uint32_t)last_phase[s], a.status, 743, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        constexpr uint32_t idesc = mx_idesc(128, NT);
        const uint32_t leader = elect_one();
        const uint32_t tbase = __shfl_sync(0xffffffffu, tmem_base, 0);
        const int tiles = __shfl_sync(0xffffffffu, total, 0);
        const uint32_t s_stages = __shfl_sync(0xffffffffu, smem_u32(stages), 0);
        const uint32_t s_scales = __shfl_sync(0xffffffffu, smem_u32(scales), 0);
        const uint32_t s_empty = __shfl_sync(0xffffffffu, smem_u32(&m->empty[0]), 0);
        const uint32_t s_sempty = __shfl_sync(0xffffffffu, smem_u32(&m->sempty[0]), 0);
        const uint32_t s_tfull = __shfl_sync(0xffffffffu, smem_u32(&m->tfull[0]), 0);
        int stage = 0, acc = 0, slot = 0, in_slot = 0;
        uint32_t phase = 0, acc_phase = 0, sphase = 0;
        bool ok = true;
        for (int t = unit; t < tiles && ok; t += units) {
            if (!warp_wait_all(&m->tempty[acc], acc_phase ^ 1u, a.status, 744, abort_flag)) break;
            tc_fence_after();
            const uint32_t d0 = tbase + (uint32_t)(acc * 2 * NT);
            const int kb0 = 4 * first_group(t % splits), kb1 = end_kb(t % splits);
            for (int kb = kb0; kb < kb1; ++kb) {
                if ((in_slot == 0 && !warp_wait_all(&m->sfull[slot], sphase, a.status, 747, abort_flag)) ||
                    !warp_wait_all(&m->full[stage], phase, a.status, 746, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tsf = tbase + G::SF_COL + (uint32_t)((kb & 1) * SF_BUF_COLS);
                const uint64_t sdesc = scale_desc(s_scales + (uint32_t)(slot * SF_SLOT_BYTES + in_slot * SF_BYTES));
                copy_scales<false>(leader, tsf, sdesc);                     // the tokens'
                copy_scales<false>(leader, tsf + 4, sdesc + (512 >> 4));    // the weights'
                copy_scales<false>(leader, tsf + 8, sdesc + (1024 >> 4));
                const uint64_t wdesc = umma_desc_sw128(s_stages + (uint32_t)stage * G::OP_BYTES, 16, 1024);
                const uint64_t xdesc = wdesc + (2 * G::W_BYTES >> 4);
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        mma_mx8<false>(leader, d0 + b * NT, wdesc + (b * G::W_BYTES >> 4) + kk * 2, xdesc + kk * 2,
                                       idesc | ((uint32_t)kk << 4) | ((uint32_t)kk << 29), tsf + 4 + 4 * b, tsf,
                                       kk != 0 ? 1u : (kb != kb0 ? 1u : 0u));
                commit<false>(leader, s_empty + (uint32_t)stage * 8);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++in_slot == SF_GROUP || kb == kb1 - 1) {
                    commit<false>(leader, s_sempty + (uint32_t)slot * 8);
                    in_slot = 0;
                    if (++slot == SF_SLOTS) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                }
            }
            if (!ok) break;
            commit<false>(leader, s_tfull + (uint32_t)acc * 8);
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        __syncwarp();
        if (leader) umma_commit(&m->drain);
        __syncwarp();
        warp_wait_all(&m->drain, 0, a.status, 748, nullptr);
    } else if (warp < EPI_WARP0) {
        // ------------------------------------------------ scales
        const int i = (warp - 2) * 32 + lane;
        const int nb = a.Kdim / kMxBlock;
        const uint32_t off = (uint32_t)((i & 31) * 16 + (i >> 5) * 4);
        const uint8_t *px = nullptr, *pw0 = nullptr, *pw1 = nullptr;
        auto rows_of = [&](int t) {
            int e, m_row0, row_end, n0;
            decode_tile(m, E, NT, BN, t / splits, e, m_row0, row_end, n0);
            const int64_t row = (int64_t)m_row0 + i;
            px = i < NT && row < row_end ? a.as + row * nb : nullptr;
            const int n = n0 + i, n2 = GATEUP ? n : n + 128;
            const int64_t be = (int64_t)e * a.N;
            pw0 = n < a.N ? a.b0s + (be + n) * nb : nullptr;
            pw1 = n2 < a.N ? (GATEUP ? a.b1s : a.b0s) + (be + n2) * nb : nullptr;
        };
        uint4 vx[2], v0[2], v1[2];
        int ld_t = unit, ld_g = unit < total ? first_group(unit % splits) : 0;
        bool fresh = true;
        auto load_weights = [&](int i2) {
            v0[i2] = load_scales<true>(pw0, ld_g, nb);
            v1[i2] = load_scales<true>(pw1, ld_g, nb);
        };
        auto load_tokens = [&](int i2) { vx[i2] = load_scales<false>(px, ld_g, nb); };
        auto load_next = [&](int i2) {
            if (ld_t >= total) return;
            if (fresh) rows_of(ld_t);
            load_weights(i2);
            load_tokens(i2);
            fresh = 4 * ++ld_g >= end_kb(ld_t % splits);
            if (fresh) {
                ld_t += units;
                ld_g = first_group(ld_t % splits);
            }
        };
        if (!GATEUP) asm volatile("griddepcontrol.wait;" ::: "memory");
        load_next(0);
        load_next(1);
        int slot = 0;
        uint32_t sphase = 0;
        int64_t mine = 0;  // this CTA's groups
        for (int t = unit; t < total; t += units)
            mine += (end_kb(t % splits) + 3) / 4 - first_group(t % splits);
        for (int64_t n = 0; n < mine; n += 2) {
            bool ok = true;
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
                if (n + i2 >= mine) break;
                if (!warp_wait(&m->sempty[slot], sphase ^ 1u, lane, a.status, 749, abort_flag)) {
                    ok = false;
                    break;
                }
                uint8_t* dst = scales + (size_t)slot * SF_SLOT_BYTES + off;
#pragma unroll
                for (int k = 0; k < SF_GROUP; ++k) {
                    *reinterpret_cast<uint32_t*>(dst + k * SF_BYTES) = word_of(vx[i2], k);
                    *reinterpret_cast<uint32_t*>(dst + k * SF_BYTES + 512) = word_of(v0[i2], k);
                    *reinterpret_cast<uint32_t*>(dst + k * SF_BYTES + 1024) = word_of(v1[i2], k);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m->sfull[slot]);
                if (++slot == SF_SLOTS) {
                    slot = 0;
                    sphase ^= 1u;
                }
                load_next(i2);
            }
            if (!ok) break;
        }
    } else {
        // ------------------------------------------------ epilogue: lane = weight row
        const int quad = warp & 3;
        const int half = (warp - EPI_WARP0) >> 2;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int t = unit; t < total; t += units) {
            int e, m_row0, row_end, n0;
            decode_tile(m, E, NT, BN, t / splits, e, m_row0, row_end, n0);
            const int rows = row_end - m_row0 < NT ? row_end - m_row0 : NT;
            float w = 1.f;  // lane j: token j's weight
            if (!GATEUP && !CUT && a.perm != nullptr && lane < rows) {
                const int32_t pa = a.perm[m_row0 + lane];
                w = 0.f;
                if (pa >= 0 && (int64_t)pa < a.nk) w = a.topk_w[pa];
                else if (half == 0) raise_flag(a.status, kFlagBounds, 741);
            }
            if (!warp_wait(&m->tfull[acc], acc_phase, lane, a.status, 750, abort_flag)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * 2 * NT);
            if (GATEUP) {  // this half's tokens
                constexpr int H = NT / 2;
                uint32_t g[H], u[H];
                tmem_ld<H>(taddr + half * H, g);
                tmem_ld<H>(taddr + NT + half * H, u);
                tmem_ld_wait();
                const int f0 = n0 + quad * 32;
                if (f0 < a.N) {
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const int r = half * H + j;
                        if (r >= rows) break;
                        const float h = swiglu(__uint_as_float(g[j]), __uint_as_float(u[j]));
                        const uint32_t b = mx_scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(h)));
                        const int64_t row = (int64_t)m_row0 + r;
                        a.h[row * a.N + f0 + lane] = (uint8_t)mx_pack4(h, 0.f, 0.f, 0.f, mx_inv_scale(b));
                        if (lane == 0) a.hs[row * (a.N / kMxBlock) + f0 / kMxBlock] = (uint8_t)b;
                    }
                }
            } else {  // this half's 128 rows of D
                uint32_t v[NT];
                tmem_ld<NT>(taddr + half * NT, v);
                tmem_ld_wait();
                const int d0 = n0 + half * 128 + quad * 32;
                if (d0 < a.N) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (j >= rows) break;
                        if (CUT) {
                            a.part[((int64_t)(t % splits) * a.max_rows + m_row0 + j) * a.N + d0 + lane] =
                                __uint_as_float(v[j]);
                            continue;
                        }
                        const float wj = __shfl_sync(0xffffffffu, w, j);
                        a.y[((int64_t)m_row0 + j) * a.N + d0 + lane] = __float2bfloat16_rn(wj * __uint_as_float(v[j]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->tempty[acc]);
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, G::TMEM);
    }
}

// y = bf16(w (part 0 + part 1 + ...)), in that order: the rows of a down product whose
// contracted axis was cut.  A thread per 4 elements.
__global__ void __launch_bounds__(256) ffn_mx8_join_kernel(const Args a)
{
    bool bad = false;
    for (int e = threadIdx.x; e < a.E; e += 256) {
        const int r0 = a.offsets[e], r1 = a.offsets[e + 1];
        bad |= r0 < 0 || r1 < r0 || (int64_t)r1 > a.max_rows;
    }
    if (__syncthreads_or(bad)) return;  // nothing was computed (the products raised the flag)
    const int64_t row = blockIdx.y;
    if (row < a.offsets[0] || row >= a.offsets[a.E]) return;
    float w = 1.f;
    if (a.perm != nullptr) {
        const int32_t pa = a.perm[row];
        w = 0.f;
        if (pa >= 0 && (int64_t)pa < a.nk) w = a.topk_w[pa];
        else if (blockIdx.x == 0 && threadIdx.x == 0) raise_flag(a.status, kFlagBounds, 751);
    }
    const int d = 4 * (int)(blockIdx.x * 256 + threadIdx.x);
    if (d >= a.N) return;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int sp = 0; sp < a.splits; ++sp) {
        const float4 v = *reinterpret_cast<const float4*>(a.part + ((int64_t)sp * a.max_rows + row) * a.N + d);
        t.x += v.x;
        t.y += v.y;
        t.z += v.z;
        t.w += v.w;
    }
    *reinterpret_cast<uint2*>(a.y + row * a.N + d) = make_uint2(pack_bf16x2(w * t.x, w * t.y), pack_bf16x2(w * t.z, w * t.w));
}

// ------------------------------------------------------------------- host --
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encoder()
{
    static std::atomic<EncodeTiledFn> cached{nullptr};
    EncodeTiledFn fn = cached.load(std::memory_order_acquire);
    if (fn == nullptr) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<EncodeTiledFn>(p);
            cached.store(fn, std::memory_order_release);
        }
    }
    return fn;
}

// Row-major bytes (.., rows, K), read in boxes of box_rows x 128 with the
// 128-byte swizzle; E = 0: two dimensions.
static bool map_bytes(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint64_t E, uint32_t box_rows)
{
    EncodeTiledFn enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {K, rows, E};
    cuuint64_t strides[2] = {K, K * rows};
    cuuint32_t box[3] = {BK, box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, E ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y (rows, cols) bf16 for stores of 32 rows x 64 columns from shared memory laid out
// with the 128-byte swizzle.
static bool map_store(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows)
{
    EncodeTiledFn enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * 2};
    cuuint32_t box[2] = {64, 32};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Per device: shared memory opted in, and how many CTAs or pairs are resident.
template <bool GATEUP, bool PAIR> static cudaError_t prepare(int* resident)
{
    static std::atomic<int> cached[32];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 32) {
        const int v = cached[dev].load(std::memory_order_acquire);
        if (v > 0) {
            *resident = v;
            return cudaSuccess;
        }
    }
    constexpr size_t smem = smem_bytes<GATEUP, PAIR>();
    e = cudaFuncSetAttribute(ffn_mx8_kernel<GATEUP, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int units = 0;
    if (PAIR) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(NUM_THREADS, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&units, ffn_mx8_kernel<GATEUP, PAIR>, &cfg);
    } else {
        e = cudaDeviceGetAttribute(&units, cudaDevAttrMultiProcessorCount, dev);  // one CTA per SM
    }
    if (e != cudaSuccess) return e;
    if (units < 1) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 32) cached[dev].store(units, std::memory_order_release);
    *resident = units;
    return cudaSuccess;
}

template <bool GATEUP, bool PAIR>
static cudaError_t launch_one(const CUtensorMap& mA, const CUtensorMap& mB0, const CUtensorMap& mB1,
                              const CUtensorMap& mY, const Args& a, int64_t tiles_bound, cudaStream_t s)
{
    int units = 0;
    cudaError_t e = prepare<GATEUP, PAIR>(&units);
    if (e != cudaSuccess) return e;
    int64_t n = tiles_bound < units ? tiles_bound : units;
    if (n < 1) n = 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (PAIR) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = 2;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    if (!GATEUP) {  // may start before the gate/up product has ended
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.gridDim = dim3((unsigned)(Geo<GATEUP, PAIR>::CTAS * n), 1, 1);
    cfg.blockDim = dim3(NUM_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<GATEUP, PAIR>();
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, ffn_mx8_kernel<GATEUP, PAIR>, mA, mB0, mB1, mY, a);
}

template <bool GATEUP, int NT, bool CUT>
static cudaError_t launch_few(const CUtensorMap& mX, const CUtensorMap& mW0, const CUtensorMap& mW1, const Args& a,
                              int64_t tiles_bound, cudaStream_t s)
{
    static PerDeviceFlag opted;
    int dev = 0, sms = 0;
    cudaError_t e = opt_in_smem(opted, reinterpret_cast<const void*>(ffn_mx8_few_kernel<GATEUP, NT, CUT>), Few<NT>::SMEM);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(tiles_bound < sms ? tiles_bound : sms), 1, 1);
    cfg.blockDim = dim3(NUM_THREADS, 1, 1);
    cfg.dynamicSmemBytes = Few<NT>::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = GATEUP ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, ffn_mx8_few_kernel<GATEUP, NT, CUT>, mX, mW0, mW1, a);
}

}  // namespace mx

// Tiles of few rows there can be, for n_tiles tiles along the product's columns.
static int64_t few_tiles(const moe_config& c, int64_t max_rows, int n_tiles)
{
    const int64_t m = c.E + max_rows / 32;
    return (max_rows < m ? max_rows : m) * n_tiles;
}

// Parts the down product's contracted axis is cut in: with few tokens its tiles leave
// most SMs without a stream of weights.  (One token, 2 of 8 experts, D = 4096,
// F = 14336: both products 90 us with 32 tiles for 148 SMs, 70 with each in four
// parts and a kernel that joins them.)
static int few_splits(const moe_config& c, int64_t max_rows)
{
    if (max_rows > mx::kFewRows * (int64_t)c.E) return 1;
    const int64_t tiles = few_tiles(c, max_rows, (c.D + 255) / 256), groups = (c.F + 511) / 512;
    int64_t n = 148 / tiles;
    if (n > 8) n = 8;
    // two groups of four stages each at least (D = 2048, F = 1408, 6 of 64 experts: 22.5 us
    // whole, 23.6 in three parts of one group)
    if (n > groups / 2) n = groups / 2;
    return n > 1 ? (int)n : 1;
}

// Scratch for the parts of every number of rows up to max_rows, so that a workspace of
// a larger batch serves a smaller one: n parts are cut for at most the rows whose tiles,
// min(rows, E + rows / 32) n_tiles, fit 148 / n times.
size_t mx8_part_bytes(const moe_config& c, int64_t max_rows)
{
    const int64_t n_tiles = (c.D + 255) / 256, most = ((c.F + 511) / 512) / 2 < 8 ? ((c.F + 511) / 512) / 2 : 8;
    const int64_t few = max_rows < mx::kFewRows * (int64_t)c.E ? max_rows : mx::kFewRows * (int64_t)c.E;
    int64_t rows = 0;  // the most of n times its rows
    for (int64_t n = 2; n <= most; ++n) {
        const int64_t q = 148 / n / n_tiles;
        const int64_t fit = q < c.E ? q : 32 * (q - c.E) + 31 > q ? 32 * (q - c.E) + 31 : q;
        const int64_t r = fit < few ? fit : few;
        if (n * r > rows) rows = n * r;
    }
    return (size_t)rows * c.D * sizeof(float);
}

cudaError_t launch_ffn_mx8(const moe_config& c, int64_t max_rows, const void* xq, const void* xs,
                           const int32_t* offsets, const int32_t* perm, const float* topk_w,
                           const moe_mx8_weights& w, void* hq, void* hs, void* y_perm, void* amaps, void* part,
                           int* status, cudaStream_t s)
{
    using namespace mx;
    auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
    const uint64_t D = (uint64_t)c.D, F = (uint64_t)c.F, E = (uint64_t)c.E, R = (uint64_t)max_rows;
    Args a{};
    a.offsets = offsets; a.perm = perm; a.topk_w = topk_w;
    a.as = u8(xs); a.b0s = u8(w.gate_scales); a.b1s = u8(w.up_scales);
    a.h = static_cast<uint8_t*>(hq); a.hs = static_cast<uint8_t*>(hs);
    a.E = c.E; a.Kdim = c.D; a.N = c.F; a.n_tiles = (c.F + 127) / 128;
    a.max_rows = max_rows; a.nk = c.T * c.K; a.status = status;
    Args d = a;  // the down product
    d.as = u8(hs); d.b0s = d.b1s = u8(w.down_scales);
    d.y = static_cast<__nv_bfloat16*>(y_perm);
    d.Kdim = c.F; d.N = c.D; d.n_tiles = (c.D + 255) / 256;
    CUtensorMap mX, mG, mU, mH, mD, mY;
    if (max_rows <= kFewRows * (int64_t)c.E) {
        constexpr int NT = 32;
        if (!map_bytes(&mX, xq, D, R, 0, NT) || !map_bytes(&mG, w.gate, D, F, E, 128) ||
            !map_bytes(&mU, w.up, D, F, E, 128) || !map_bytes(&mH, hq, F, R, 0, NT) ||
            !map_bytes(&mD, w.down, F, D, E, 128))
            return cudaErrorInvalidValue;
        a.splits = 1;
        d.splits = few_splits(c, max_rows);
        d.part = static_cast<float*>(part);
        cudaError_t e = launch_few<true, NT, false>(mX, mG, mU, a, few_tiles(c, max_rows, a.n_tiles), s);
        if (e != cudaSuccess) return e;
        const int64_t tiles = few_tiles(c, max_rows, d.n_tiles);
        if (d.splits == 1) return launch_few<false, NT, false>(mH, mD, mD, d, tiles, s);
        e = launch_few<false, NT, true>(mH, mD, mD, d, tiles * d.splits, s);
        if (e != cudaSuccess) return e;
        ffn_mx8_join_kernel<<<dim3((unsigned)((c.D + 1023) / 1024), (unsigned)max_rows), 256, 0, s>>>(d);
        return cudaGetLastError();
    }
    if (!map_bytes(&mX, xq, D, R, 0, 128) || !map_bytes(&mG, w.gate, D, F, E, 64) ||
        !map_bytes(&mU, w.up, D, F, E, 64) || !map_bytes(&mH, hq, F, R, 0, 128) ||
        !map_bytes(&mD, w.down, F, D, E, 64) || !map_store(&mY, y_perm, D, R))
        return cudaErrorInvalidValue;
    // CTA pairs when experts hold 128 rows or more on average, as the bf16
    // experts: single CTAs waste fewer padded rows on a few tokens each
    const bool pair = max_rows >= 128 * (int64_t)c.E;
    const int64_t bm = pair ? 256 : 128;
    const int64_t mt = (max_rows + bm - 1) / bm + c.E;
    // rows of a tile past its expert's end are not fetched: worth a launch only
    // where a tile can reach other experts' rows beyond one tile of them all
    const CUtensorMap* gm = nullptr;
    if (max_rows > 128) {
        cudaError_t e = launch_ffn_amaps(&mX, &mH, offsets, c.E, max_rows, amaps, s);
        if (e != cudaSuccess) return e;
        gm = static_cast<const CUtensorMap*>(amaps);
    }
    a.amaps = gm;
    d.amaps = gm ? gm + c.E : nullptr;
    cudaError_t e = pair ? launch_one<true, true>(mX, mG, mU, mY, a, mt * a.n_tiles, s)
                         : launch_one<true, false>(mX, mG, mU, mY, a, mt * a.n_tiles, s);
    if (e != cudaSuccess) return e;
    return pair ? launch_one<false, true>(mH, mD, mD, mY, d, mt * d.n_tiles, s)
                : launch_one<false, false>(mH, mD, mD, mY, d, mt * d.n_tiles, s);
}

}  // namespace moe
