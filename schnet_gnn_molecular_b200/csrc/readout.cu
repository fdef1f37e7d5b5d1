// Readout tuning from stored features: the 8-bit store, readout energies and the
// readout's weight gradients (no counterpart on the pages; the readout is the model's
// eps = ssp(x R1 + c1) R2 + c2, hidden width H = F/2).
//
// Store: per row (at most 128 features, one block) the scale is a power of two, so
// x / scale is exact and the e4m3 rounding is the only one: codes are a function of
// x alone, whatever computes them.  It is bound by HBM: 641 bytes a float32 row of 128,
// 10^6 rows in 107 us on the device (92 % of a copy's rate), 117 a call back to back.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cuda.h>
#include <cuda_fp8.h>

#include "internal.h"

namespace schnet {

// ---------------------------------------------------------------------------
// 8-bit feature store
// ---------------------------------------------------------------------------
constexpr int ST = 256;                  // threads per CTA
constexpr int STORE_ROWS = 4;            // rows a warp has in flight

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// scale byte (e + 127) of a row whose largest |x| has the bits `top`: e = k - 8 for
// top = m 2^k with m <= 1.75 (448 = 1.75 * 2^8), else k - 7; 255 for NaN, infinities
// and magnitudes of 2^127 or more (their stored value could round to infinity)
__device__ __forceinline__ int scale_byte(uint32_t top)
{
    if (top >= 0x7f000000u) return 255;
    const int e = (int)(top >> 23) - 127 - ((top & 0x7fffffu) > 0x600000u ? 7 : 8);
    return max(e, -100) + 127;
}

// A warp per row, four features a lane, STORE_ROWS rows loaded before the first is
// used.  VEC: rows start on a 4-element boundary, so a lane's four come in one load.
template <class T, bool VEC>
__global__ void __launch_bounds__(ST) k_store_features(const T* __restrict__ x, long long n, int F, long long stride,
                                                       const int32_t* __restrict__ to, int W,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales)
{
    const int lane = threadIdx.x & 31, f0 = lane * 4;
    const long long warp = ((long long)blockIdx.x * ST + threadIdx.x) >> 5, nwarp = ((long long)gridDim.x * ST) >> 5;
    for (long long i0 = warp * STORE_ROWS; i0 < n; i0 += nwarp * STORE_ROWS) {
        float v[STORE_ROWS][4];
#pragma unroll
        for (int r = 0; r < STORE_ROWS; ++r) {
            const T* p = x + (i0 + r) * stride + f0;
            const bool row = i0 + r < n;
            if (VEC && row && f0 + 4 <= F) {
                struct alignas(4 * sizeof(T)) Four { T e[4]; };
                const Four q = *reinterpret_cast<const Four*>(p);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[r][k] = to_f32(q.e[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[r][k] = row && f0 + k < F ? to_f32(p[k]) : 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < STORE_ROWS; ++r) {
            uint32_t top = 0;            // |x| as bits: ordered like the values, NaN above all
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(v[r][k]) & 0x7fffffffu);
            const int b = scale_byte(__reduce_max_sync(0xffffffffu, top));
            uint32_t q = 0;
            if (b != 255) {
                const float inv = __uint_as_float((uint32_t)(254 - b) << 23);      // 2^-e
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[r][0] * inv, v[r][1] * inv),
                                                             __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[r][2] * inv, v[r][3] * inv),
                                                             __NV_SATFINITE, __NV_E4M3);
                q = lo | hi << 16;
            }
            if (i0 + r < n) {
                const long long o = to ? (long long)__ldg(to + i0 + r) : i0 + r;
                if (f0 < W) *reinterpret_cast<uint32_t*>(codes + o * W + f0) = q;
                if (lane == 0) scales[o] = (uint8_t)b;
            }
        }
    }
}

template <class T>
static cudaError_t store_launch(const void* x, long long n, int F, long long stride, const int32_t* to,
                                uint8_t* codes, uint8_t* scales, cudaStream_t s)
{
    const int W = (F + 15) / 16 * 16;
    if (n == 0) return cudaSuccess;
    const long long per = ST / 32 * STORE_ROWS;
    const unsigned grid = (unsigned)std::min<long long>((n + per - 1) / per, 148 * 8);
    const bool vec = stride % 4 == 0 && (uintptr_t)x % (4 * sizeof(T)) == 0;
    if (vec)
        k_store_features<T, true><<<grid, ST, 0, s>>>((const T*)x, n, F, stride, to, W, codes, scales);
    else
        k_store_features<T, false><<<grid, ST, 0, s>>>((const T*)x, n, F, stride, to, W, codes, scales);
    return cudaGetLastError();
}

cudaError_t launch_get_features(schnet_ctx* c, uint8_t* codes, uint8_t* scales)
{
    c->launches += 1;
    return store_launch<float>(c->ws.x, c->N, c->F, FP, c->ws.perm, codes, scales, c->s);
}

// ---------------------------------------------------------------------------
// readout energies
// ---------------------------------------------------------------------------
constexpr int MAX_SM = 256;              // status words: one per CTA, one per thread of the kernels that sum
constexpr int MAX_ATOMS = 0x7fff0000;    // row indexes a little past the last one stay in 32 bits

struct ReadoutArgs {
    const uint8_t *codes, *scales;
    int n, F, H, W, R;
    const int32_t* off;
    const float *R1, *c1, *R2, *c2;
    float *energy, *eps;
    double* csum;                        // [ceil(n / 32)] sums of 32 atoms' eps
    uint32_t* status;                    // [CTAs] 1: a device-side wait gave up
    int ncta;
    const float* gE;
    float *dR1, *dc1, *dR2, *dc2;
    float* part;                         // [CTAs][64 h][128 f] sums of D2
    int nseed;                           // CTAs of the seeds kernel
    float* gat;                          // [n up to a multiple of 4] g of each atom
    double* part2;                       // [nseed] shares of dc2
    double* colpart;                     // [CTAs][128] column sums of 2 g sigma, g ssp / ln2
};

__device__ __forceinline__ int off_at(const ReadoutArgs& a, int r) { return min(max(__ldg(a.off + r), 0), a.n); }

// x^L tiles come by TMA: 128 rows of 128 bytes, 128-byte swizzled (16-byte piece c of
// row r lies at piece c ^ (r & 7)), so that a warp whose lanes each read their own row
// meets every bank once per 8 lanes.  Columns past W and rows past n read as zero.
constexpr uint32_t TILE_BYTES = 128 * 128;
constexpr uint32_t RO_POLLS = 1u << 22;

__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int row, uint64_t* bar)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(TILE_BYTES)
                 : "memory");
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(0), "r"(row), "r"(smem_u32(bar))
                 : "memory");
}

// two e4m3 codes -> fp16 pair (exact)
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// 16 consecutive 32-bit TMEM columns of this warp's 32 lanes <- 16 registers per thread
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// N consecutive TMEM columns of this warp's 32 lanes -> N registers per thread
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[N])
{
    if constexpr (N == 32) {
        tmem_ld32(taddr, r);
    } else if constexpr (N == 16) {
        tmem_ld16(taddr, r);
    } else {
        static_assert(N == 8, "8, 16 or 32 columns");
        uint32_t* u = reinterpret_cast<uint32_t*>(r);
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                     : "r"(taddr));
    }
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One lane of a converged warp.  The MMAs below are issued by a whole warp with a predicate
// from here and warp-uniform operands: behind a branch on the thread index the compiler
// moves every operand to a uniform register anew, which costs 60-130 cycles an MMA against 20.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p;
}

// D[tmem] (+)= A[tmem] B[smem desc] and D[tmem] (+)= A[smem desc] B[smem desc], kind::f16,
// by the lane with go != 0
__device__ __forceinline__ void mma_ts(uint32_t go, uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"(acc), "r"(go)
                 : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t go, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(acc), "r"(go)
                 : "memory");
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// R1 as the MMA's B operand [64 h][128 f] (K-major core matrices), two fp16 terms of
// R1 2^s with 2^s the power of two that brings the largest |R1| to [2^14, 2^15): hi + lo
// carry 22 bits, and entries 2^-24 of the largest still lose nothing above 2^-39 of it.
// Returns 2^-s, or NaN where R1 or c1 holds a NaN or an infinity (in the accumulators it would
// reach only its own hidden unit); red: one word per warp.
constexpr uint32_t R1_TERM = HP * FP * 2;
template <int THREADS>
struct StageR1 {
    static constexpr int PAIRS = (HP * FP / 2 + THREADS - 1) / THREADS;   // (f, f + 1) of one hidden unit each
    float v[PAIRS][2];
    uint32_t mx;                                                // as bits, which order like the magnitudes

    // the loads, first thing in the kernel: what follows hides their latency
    __device__ __forceinline__ explicit StageR1(const ReadoutArgs& a)
    {
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            const int k = threadIdx.x + j * THREADS, h = k % HP, f = k / HP * 2;
#pragma unroll
            for (int u = 0; u < 2; ++u) v[j][u] = h < a.H && f + u < a.F ? __ldg(a.R1 + (f + u) * a.H + h) : 0.f;
        }
        mx = threadIdx.x < a.H ? __float_as_uint(__ldg(a.c1 + threadIdx.x)) : 0u;
    }

    // a barrier of the whole CTA inside
    __device__ __forceinline__ float store(uint8_t* hi, uint8_t* lo, uint32_t* red)
    {
        mx = (mx & 0x7fffffffu) >= 0x7f800000u ? 0x7f800000u : 0u;
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
            mx = max(mx, max(__float_as_uint(v[j][0]) & 0x7fffffffu, __float_as_uint(v[j][1]) & 0x7fffffffu));
        mx = __reduce_max_sync(0xffffffffu, mx);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
        __syncthreads();
        mx = (threadIdx.x & 31) < THREADS / 32 ? red[threadIdx.x & 31] : 0u;
        mx = __reduce_max_sync(0xffffffffu, mx);
        const int ex = (int)(mx >> 23);
        const int s = ex > 0 && ex < 255 ? min(110, 14 - (ex - 127)) : 0;       // -113 .. 110: 2^s and 2^-s are normal
        const float up = __uint_as_float((uint32_t)(127 + s) << 23);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            const int k = threadIdx.x + j * THREADS, h = k % HP, f = k / HP * 2;
            if (k >= HP * FP / 2) break;
            uint32_t vh, vl;
            split2<0>(v[j][0] * up, v[j][1] * up, vh, vl);
            *reinterpret_cast<uint32_t*>(hi + kmajor_off(h, f, HP)) = vh;
            *reinterpret_cast<uint32_t*>(lo + kmajor_off(h, f, HP)) = vl;
        }
        return ex == 255 ? __int_as_float(0x7fffffff) : __uint_as_float((uint32_t)(127 - s) << 23);
    }
};

// log2((1 + 2^t) / 2) for |t| <= 3 as t / 2 and an even polynomial (ssp2_fit.py; relative error 2e-7),
// for a warp's units whose t are all this small; which they are is looked at 8 at a time.
// The MUFU logarithm errs by up to 2^-22 around 1 and by 6e-8 on average, the same way for every
// atom: with it alone the energies of 64 chains are off by 2-7e-6, 2-5e-5 and 1-7e-4 of themselves
// at a tenth, hundredth and thousandth of Xavier weights, dR2 by 6e-6, 4e-5 and 8e-4; with this
// both by 1-3e-7 (torch's float32 forms: energies 4-9e-7, 3e-6, 3-9e-5, dR2 6e-7, 3e-6, 7e-5).
constexpr float SSP2_SMALL = 3.f;
__device__ __forceinline__ float2 ssp2_small(float2 t)
{
    const float2 s = mul2(t, t);
    float2 q = fma2(dup2(-1.0950124140762796e-09f), s, dup2(6.010890274410485e-08f));
    q = fma2(q, s, dup2(-1.9344583961355966e-06f));
    q = fma2(q, s, dup2(5.532750947168097e-05f));
    q = fma2(q, s, dup2(-0.0017342476639896631f));
    q = fma2(q, s, dup2(0.08664331585168839f));
    return mul2(t, fma2(t, q, dup2(0.5f)));
}

// the factor that takes an accumulator of row i (codes times R1 2^s) to p log2(e)
__device__ __forceinline__ float row_factor(int byte, float down)
{
    if (byte == 255 || down != down) return __int_as_float(0x7fffffff);
    return fminf(__uint_as_float((uint32_t)byte << 23) * down, 1e38f) * LOG2EF;
}

// E_r: TPR threads add the sums of the 32-atom chunks inside the replica and the single
// atoms at its ends, in float64 and a fixed order; the sum is lane 0's of each warp.
template <int TPR>
__device__ __forceinline__ double replica_sum(const ReadoutArgs& a, int r, int l)
{
    double s = 0.0;
    const int lo = off_at(a, r), hi = off_at(a, r + 1);
    const int c0 = (lo + 31) >> 5, c1 = hi >> 5;                 // whole chunks [c0, c1)
    if (c0 < c1) {
        for (int i = lo + l; i < c0 * 32; i += TPR) s += (double)a.eps[i];
        for (int c = c0 + l; c < c1; c += TPR) s += a.csum[c];
        for (int i = c1 * 32 + l; i < hi; i += TPR) s += (double)a.eps[i];
    } else {
        for (int i = lo + l; i < hi; i += TPR) s += (double)a.eps[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Energies.  Three groups of 8 warps and one issuing warp share the CTA's R1.  A group takes
// every (3 gridDim)-th tile of 128 atoms, a thread one atom and half of its hidden units:
// half its row of codes is read from the TMA stage, widened to fp16 (exact) and put into
// tensor memory as the MMA's A operand (lane = atom), so D[atom][h] = codes . R1 comes back
// with 32 hidden units per thread; the halves meet through shared memory, on two barriers in
// turn (the upper half may finish a tile ahead of the lower, not two: the next MMAs wait for
// both).  A group widens tile it+1, reads D(it) into registers, hands both on to the issuing
// warp and only then works on D(it), which hides the MMAs.  The issuing thread blocks while
// the tensor core's queue is full, so it does nothing else.
// Bound: 2 transcendentals per hidden unit on the MUFU, 8 cycles an atom and SM (HBM: 133
// bytes, 5.9 cycles; MMAs: 4).  4.2 M atoms: 187 us in short runs, 222 for seconds on end (the
// power cap).  Tried, in short runs against 180 before the small units had their polynomial:
// exponentials on the FMA pipe (one pair in 8, 4, 2) cost more issue slots than they free on the
// MUFU, 180, 186, 192 us; one thread per atom with four groups of 4 warps (96 registers) 195;
// widening warps apart, D doubled (64 registers) 176 us for 171, and 1 us more for small calls.
// 269 atoms: 8.0 us with the sums' kernel.
// The look whether 8 units are all small (ssp2_small) costs 5 % at 4.2 M atoms, so a warp takes it at
// every 8th tile and as long as it finds any: 218 us for 217 without it.  So an atom's eps may
// differ by that polynomial's rounding with the atoms that share its warp, not from call to call.
// FW is the width that codes and hidden layer are padded to: 64 up to 64 features (a thread
// has 32 codes and 16 units, the MMAs half their K and N), else 128.  At 64 features the
// 64 form takes 117 us for 4.2 M atoms against 187 of the 128 form, and 15.9 against 20.5 for
// 192,000; the same choice made at run time inside one kernel cost 128 features 14 %.
constexpr int FWD_GROUPS = 3, FWD_STAGES = 3, FWD_GT = 256, FWD_THREADS = FWD_GROUPS * FWD_GT + 32;
constexpr int FWD_LOOK = 8;                                      // tiles from look to look
constexpr uint32_t FWD_R1 = FWD_GROUPS * FWD_STAGES * TILE_BYTES;
constexpr uint32_t FWD_CST = FWD_R1 + 2 * R1_TERM;               // float4[32]: c1 log2e, R2 ln2 of two units
constexpr uint32_t FWD_RED = FWD_CST + 32 * 16;
constexpr uint32_t FWD_EX = FWD_RED + 128;                       // per group: float[2][128], the upper halves' sums
constexpr uint32_t FWD_BAR = FWD_EX + FWD_GROUPS * 2 * 128 * 4;
constexpr int FWD_NBAR = FWD_STAGES + 2 + 8;                     // per group: stages full, A ready, MMAs done, [2][4] upper sums
constexpr uint32_t FWD_SMEM = FWD_BAR + 8 * FWD_GROUPS * FWD_NBAR + 16;

template <int FW>
__global__ void __launch_bounds__(FWD_THREADS, 1)
k_readout_eps(const __grid_constant__ CUtensorMap map, ReadoutArgs a)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    float4* cst = reinterpret_cast<float4*>(sm + FWD_CST);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + FWD_BAR);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + FWD_GROUPS * FWD_NBAR);
    constexpr int HW = FW / 2, HT = HW / 2;                       // hidden units: all, and a thread's
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int ntiles = (a.n + 127) / 128, ngroups = FWD_GROUPS * gridDim.x;
    const uint32_t stages = smem_u32(sm);
    auto tiles_of = [&](int gid) { return gid < ntiles ? (ntiles - gid + ngroups - 1) / ngroups : 0; };
    auto first_row = [&](int g, int it) { return ((int)blockIdx.x + (int)gridDim.x * g + it * ngroups) * 128; };

    pdl_trigger();
    StageR1<FWD_THREADS> r1(a);
    if (warp == 0) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == FWD_GROUPS * FWD_GT) {                     // the first tiles are on their way before R1 is stored
        for (int g = 0; g < FWD_GROUPS; ++g) {
            uint64_t* full = bars + g * FWD_NBAR;
            for (int k = 0; k < FWD_STAGES; ++k) mbar_init(full + k, 1);
            mbar_init(full + FWD_STAGES, FWD_GT / 32);
            mbar_init(full + FWD_STAGES + 1, 1);
            for (int k = 0; k < 8; ++k) mbar_init(full + FWD_STAGES + 2 + k, 1);
        }
        fence_mbar_init();
        for (int it = 0; it < FWD_STAGES; ++it)
            for (int g = 0; g < FWD_GROUPS; ++g)
                if (it < tiles_of(blockIdx.x + gridDim.x * g))
                    tma_tile(stages + (g * FWD_STAGES + it) * TILE_BYTES, &map, first_row(g, it), bars + g * FWD_NBAR + it);
    }
    if (warp == 1) {
        const int k = threadIdx.x & 31, h = 2 * k;
        const bool i0 = h < a.H, i1 = h + 1 < a.H;
        cst[k] = make_float4(i0 ? __ldg(a.c1 + h) * LOG2EF : 0.f, i1 ? __ldg(a.c1 + h + 1) * LOG2EF : 0.f,
                             i0 ? __ldg(a.R2 + h) * LN2F : 0.f, i1 ? __ldg(a.R2 + h + 1) * LN2F : 0.f);
    }
    const float down = r1.store(sm + FWD_R1, sm + FWD_R1 + R1_TERM, reinterpret_cast<uint32_t*>(sm + FWD_RED));
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    bool ok = true;

    if (warp == FWD_GROUPS * FWD_GT / 32) {
        // ---- issuing warp: every group's tiles in turn
        const uint32_t id = idesc_f16(128, HW, 0, 0);
        const uint64_t bhi = smem_desc(stages + FWD_R1, HP * 16, 128);
        const uint64_t blo = smem_desc(stages + FWD_R1 + R1_TERM, HP * 16, 128);
        const uint32_t tm0 = __shfl_sync(0xffffffffu, *tslot, 0), go = elect_one();
        const int most = tiles_of(blockIdx.x);
        for (int it = 0; it < most && ok; ++it)
            for (int g = 0; g < FWD_GROUPS; ++g) {
                const int nt = tiles_of(blockIdx.x + gridDim.x * g);
                if (it >= nt) continue;
                uint64_t* full = bars + g * FWD_NBAR;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(full + FWD_STAGES, (uint32_t)it & 1u, RO_POLLS));
                if (!ok) break;
                tc_fence_after();
                const uint32_t tm = tm0 + 128 * g;
#pragma unroll
                for (int ks = 0; ks < FW / 16; ++ks)              // the small terms first
                    mma_ts(go, tm + 64, tm + ks * 8, blo + (uint64_t)((ks * 2 * HP * 16) >> 4), id, ks > 0 ? 1u : 0u);
#pragma unroll
                for (int ks = 0; ks < FW / 16; ++ks)
                    mma_ts(go, tm + 64, tm + ks * 8, bhi + (uint64_t)((ks * 2 * HP * 16) >> 4), id, 1u);
                if (go) {
                    mma_commit(full + FWD_STAGES + 1);
                    const int st = it % FWD_STAGES;               // the group has read this stage
                    if (it + FWD_STAGES < nt)
                        tma_tile(stages + (g * FWD_STAGES + st) * TILE_BYTES, &map, first_row(g, it + FWD_STAGES), full + st);
                }
                __syncwarp();
            }
        if (!ok && go)   // a wait gave up: let the copies and MMAs in flight end (bounded) before the memory goes
            for (int g = 0; g < FWD_GROUPS; ++g)
                for (int k = 0; k < FWD_STAGES + 2; ++k)
                    for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait_bounded(bars + g * FWD_NBAR + k, ph, 1u << 12);
    } else {
        const int g = threadIdx.x / FWD_GT, t = threadIdx.x & 127, half = (threadIdx.x >> 7) & 1;
        float* ex = reinterpret_cast<float*>(sm + FWD_EX) + g * 256;
        uint64_t* full = bars + g * FWD_NBAR;
        uint64_t* pair = full + FWD_STAGES + 2 + (warp & 3);      // of the two warps that share atoms
        const uint32_t tmem = *tslot + 128 * g + ((uint32_t)((warp & 3) * 32) << 16);    // A: 64 columns, D: 64 columns
        const uint32_t stage0 = stages + g * FWD_STAGES * TILE_BYTES + t * 128;
        const int nt = tiles_of(blockIdx.x + gridDim.x * g);
        const float c2 = half == 0 ? __ldg(a.c2) : 0.f;
        auto scale_of = [&](int it) {
            const int i = first_row(g, it) + t;
            return it < nt && i < a.n ? (int)__ldg(a.scales + i) : 127;
        };
        // codes of tile it -> fp16 in tensor memory, then the issuing warp's turn
        auto widen = [&](int it) {
            const int st = it % FWD_STAGES;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(full + st, (uint32_t)(it / FWD_STAGES) & 1u, RO_POLLS));
            const uint32_t src = stage0 + st * TILE_BYTES;
#pragma unroll
            for (int q = 0; q < FW / 64; ++q) {
                uint32_t v[16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 w = lds128(src + (((half * (FW / 32) + q * 2 + c) ^ (t & 7)) << 4));
                    codes_to_half(w.x, v[c * 8 + 0], v[c * 8 + 1]);
                    codes_to_half(w.y, v[c * 8 + 2], v[c * 8 + 3]);
                    codes_to_half(w.z, v[c * 8 + 4], v[c * 8 + 5]);
                    codes_to_half(w.w, v[c * 8 + 6], v[c * 8 + 7]);
                }
                tmem_st16(tmem + half * (FW / 4) + q * 16, v);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        };
        // this warp's rows are ready for the next MMAs
        auto hand_over = [&]() {
            tc_fence_before();
            __syncwarp();
            if (ok && (t & 31) == 0) mbar_arrive(full + FWD_STAGES);
        };
        bool found = false;                                       // whether the warp's last look found small units
        int byte = scale_of(0);
        if (nt > 0) {
            widen(0);
            hand_over();
        }
        for (int it = 0; it < nt && ok; ++it) {
            const float2 kk = dup2(row_factor(byte, down));
            byte = scale_of(it + 1);
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(full + FWD_STAGES + 1, (uint32_t)it & 1u, RO_POLLS));
            tc_fence_after();
            if (!ok) break;
            if (it + 1 < nt) widen(it + 1);                       // (the MMAs that read A are done)
            float d[HT];
            tmem_ld(tmem + 64 + half * HT, d);
            tmem_ld_wait();
            if (it + 1 < nt) hand_over();
            float2 e0 = make_float2(c2, 0.f), e1 = make_float2(0.f, 0.f);
            if (found || it % FWD_LOOK == 0) {
                found = false;
#pragma unroll
                for (int j0 = 0; j0 < HT / 2; j0 += 4) {              // 8 units at a time
                    float2 p[4], y[4];
                    float most = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = j0 + k;
                        const float4 c = cst[half * (HT / 2) + j];
                        p[k] = fma2(make_float2(d[2 * j], d[2 * j + 1]), kk, make_float2(c.x, c.y));
                        most = fmaxf(fmaxf(most, fabsf(p[k].x)), fabsf(p[k].y));
                    }
                    const bool small = __all_sync(0xffffffffu, most <= SSP2_SMALL);
                    found |= small && half * HT + 2 * j0 < a.H;       // (units that the layer does not have are 0)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[k] = fma2(dup2(0.5f), make_float2(ex2_mufu(-fabsf(p[k].x)), ex2_mufu(-fabsf(p[k].y))),
                                    dup2(0.5f));
                    auto sums = [&](auto poly) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float4 c = cst[half * (HT / 2) + j0 + k];
                            const float2 r2 = make_float2(c.z, c.w);
                            if (poly) {
                                e0 = fma2(r2, ssp2_small(p[k]), e0);
                            } else {
                                e0 = fma2(r2, make_float2(lg2_mufu(y[k].x), lg2_mufu(y[k].y)), e0);
                                e1 = fma2(r2, make_float2(max_nan(p[k].x, 0.f), max_nan(p[k].y, 0.f)), e1);
                            }
                        }
                    };
                    if (small) sums(std::true_type{});
                    else sums(std::false_type{});
                }
            } else {
#pragma unroll
                for (int j = 0; j < HT / 2; ++j) {
                    const float4 c = cst[half * (HT / 2) + j];
                    const float2 p = fma2(make_float2(d[2 * j], d[2 * j + 1]), kk, make_float2(c.x, c.y));
                    const float2 u = make_float2(ex2_mufu(-fabsf(p.x)), ex2_mufu(-fabsf(p.y)));
                    const float2 y = fma2(dup2(0.5f), u, dup2(0.5f));
                    e0 = fma2(make_float2(c.z, c.w), make_float2(lg2_mufu(y.x), lg2_mufu(y.y)), e0);
                    e1 = fma2(make_float2(c.z, c.w), make_float2(max_nan(p.x, 0.f), max_nan(p.y, 0.f)), e1);
                }
            }
            const int i = first_row(g, it) + t;
            float e = (e0.x + e0.y) + (e1.x + e1.y);
            if (half == 1) {
                ex[(it & 1) * 128 + t] = e;
                __syncwarp();
                if ((t & 31) == 0) mbar_arrive(pair + (it & 1) * 4);
            } else {
                ok &= __all_sync(0xffffffffu, mbar_wait_bounded(pair + (it & 1) * 4, (uint32_t)(it >> 1) & 1u, RO_POLLS));
                e += ex[(it & 1) * 128 + t];
                if (i < a.n) a.eps[i] = e;
                double s = i < a.n ? (double)e : 0.0;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if ((t & 31) == 0 && i < a.n) a.csum[i >> 5] = s;
            }
        }
    }
    tc_fence_before();
    const int gave_up = __syncthreads_or(!ok);
    if (threadIdx.x == 0) a.status[blockIdx.x] = gave_up ? 1u : 0u;
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(*tslot, 512);
    }
}

// The replicas' energies: a warp each, or a CTA where replicas are long.  Where a CTA of the
// kernel before gave up, every result is NaN, eps too (the rows it did not reach hold nothing).
template <int TPR>
__global__ void __launch_bounds__(256) k_readout_sums(ReadoutArgs a)
{
    pdl_wait();
    uint32_t bad = (int)threadIdx.x < a.ncta ? a.status[threadIdx.x] : 0u;
    const int r = TPR == 256 ? (int)blockIdx.x : (int)(blockIdx.x * (256 / TPR) + threadIdx.x / TPR);
    const int l = threadIdx.x % TPR;
    double s = r < a.R ? replica_sum<TPR>(a, r, l) : 0.0;
    __shared__ double ws[8];
    if (TPR == 256 && (threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = s;
    bad = __syncthreads_or((int)bad);
    if (TPR == 256) {
        s = 0.0;
        for (int w = 0; w < 8; ++w) s += ws[w];
    }
    if (l == 0 && r < a.R) a.energy[r] = bad ? __int_as_float(0x7fffffff) : (float)s;
    if (bad)
        for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < a.n; i += (long long)gridDim.x * 256)
            a.eps[i] = __int_as_float(0x7fffffff);
}

// a warp per replica up to 4096 atoms a replica on average, else a CTA
static schnet_status launch_sums(const ReadoutArgs& a, cudaStream_t s)
{
    const cudaError_t e = (int64_t)a.n > (int64_t)a.R * 4096
                              ? launch_pdl(k_readout_sums<256>, a.R, 256, 0, s, a)
                              : launch_pdl(k_readout_sums<32>, (a.R + 7) / 8, 256, 0, s, a);
    return enqueued(e);
}

// ---------------------------------------------------------------------------
// readout weight gradients
// ---------------------------------------------------------------------------
// A CTA takes a run of consecutive tiles.  Four widening warps turn codes into fp16, into
// tensor memory (GEMM1's A) and shared memory (GEMM2's A), and put down each row's seed
// and scale; the first of them also starts copies and MMAs.  Sixteen epilogue warps hold
// one atom and 16 hidden units a thread.  Per tile:
//   GEMM1  D1[atom][h] = codes . R1 as in the energies;
//   epilogue  per (atom, h), t = p log2(e) >= -126, y = 1/2 + 2^-t / 2: 2 sigma = 1 / y and
//     ssp(p) = ln2 (t + log2 y), which has no constant offset (small pre-activations keep
//     their bits in the sums) and for negative t keeps 2^-22 |t| absolutely (the same as the
//     rounding of t); where a warp's 8 units of 32 atoms all have |t| <= 3, a polynomial of
//     relative accuracy stands for it (finding that out costs 1.4 % at 4.2 M atoms); the
//     column sums of 2 g sigma and g ssp / ln2 stay in registers, and sigma g_i scale_i goes
//     to shared memory as an fp16 hi + residual pair;
//   GEMM2  D2[f][h] += codes^T (sigma g scale): both operands are read MN-major, so the
//     tile of codes widened once serves as it lies, and D2 stays in tensor memory from tile
//     to tile.  R2 is a factor of whole columns and is applied at the very end.
// A and D1 are doubled, X (the codes in shared memory) is held three times and B (the
// pairs) twice: every wait is for something handed over a tile earlier.
// The pair's power-of-two scale 2^E brings the largest |g_i scale_i| seen so far to
// [2^13, 2^14); when a tile has a larger one, E is lowered and the tile goes to another D2.
// The tensor core's fp32 accumulation does not round to nearest, so that happens every
// GRAD_FLUSH tiles in any case; the D2 left is emptied into fp32 sums in global memory a
// tile later, when its MMAs are long done.  The column sums are folded into float64 every
// GRAD_FOLD tiles.
// Bound: 3 transcendentals per hidden unit on the MUFU, 12 cycles an atom and SM (MMAs: 8,
// shared memory: 10, HBM: 5.8).  It takes 24: its 20 warps issue every second cycle, each
// waiting ~10 cycles an instruction (without its transcendentals 353 us for 373 at 4.2 M
// atoms, before D2 was doubled), and registers and shared memory hold no more of them.
// 4.2 M atoms: 342 us in short runs, 393 under the power cap; 545 with every warp widening its own
// rows.
// FW as in the energies: in the 64 form a thread has 8 units, GEMM2's N is 64, and what the
// unused half of X's features puts into D2 is not read.  At 64 features it takes 239 us for
// 4.2 M atoms against 342 of the 128 form, and 25 against 34 for 192,000.
constexpr int GRAD_EPI = 512, GRAD_THREADS = GRAD_EPI + 128, GRAD_XS = 3;
constexpr int GRAD_FLUSH = 8, GRAD_FOLD = 32;
constexpr uint32_t GRAD_OP = 128 * 128 * 2;                      // codes as fp16 [128][128], or [128][64 hi | 64 residual]
constexpr uint32_t GRAD_X = 2 * TILE_BYTES;
constexpr uint32_t GRAD_B = GRAD_X + GRAD_XS * GRAD_OP;
constexpr uint32_t GRAD_R1 = GRAD_B + 2 * GRAD_OP;
constexpr uint32_t GRAD_CST = GRAD_R1 + 2 * R1_TERM;             // float[64]: c1 log2e
constexpr uint32_t GRAD_RED = GRAD_CST + 64 * 4;
constexpr uint32_t GRAD_SEED = GRAD_RED + 128;                   // float[GRAD_XS][128]: the rows' seeds
constexpr uint32_t GRAD_BYTE = GRAD_SEED + GRAD_XS * 128 * 4;    // uint8[GRAD_XS][128]: their scales
constexpr uint32_t GRAD_MAX = GRAD_BYTE + GRAD_XS * 128;         // uint32[GRAD_XS][4]: largest finite |g scale| of a warp
static_assert(GRAD_MAX % 16 == 0, "read 16 bytes at a time");
constexpr uint32_t GRAD_BAR = GRAD_MAX + GRAD_XS * 16;
constexpr uint32_t GRAD_SMEM = GRAD_BAR + 8 * 10 + 16;
static_assert(GRAD_SMEM <= 227 * 1024, "one CTA's shared memory");
constexpr int PART = HP * FP;                                    // a CTA's D2 sums, [h][f]

// sums of v[0..N-1] over the warp's lanes: lane l gets column l mod N's
template <int N>
__device__ __forceinline__ float fold_columns(float (&v)[N])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = N / 2; s > 0; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int k = 0; k < s; ++k) {
            const float keep = up ? v[k + s] : v[k], send = up ? v[k] : v[k + s];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    float sum = v[0];
#pragma unroll
    for (int s = N; s < 32; s *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    return sum;
}

__device__ __forceinline__ float rcp_mufu(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Seeds: gat[i] = g of atom i's replica (0 outside all replicas), and a CTA's share of
// dc2 = sum_r g_r times the replica's atoms.  A thread takes 4 consecutive atoms: one
// bisection for the first, from there the next replica or another bisection.  Looked up
// inside the gradient kernel instead, the seeds held up its widening warps (410 us for 377
// at 4.2 M atoms) and saved 0.3 us at 269.
constexpr int SEED_ATOMS = 1024;         // atoms a CTA of 256 threads takes at a time
constexpr int MAX_SEED = 1184;           // its CTAs
__global__ void __launch_bounds__(256) k_readout_seeds(ReadoutArgs a)
{
    pdl_trigger();
    const int begin = off_at(a, 0), end = off_at(a, a.R);
    for (long long c = (long long)blockIdx.x * SEED_ATOMS; c < a.n; c += (long long)gridDim.x * SEED_ATOMS) {
        const int i0 = (int)c + threadIdx.x * 4;
        if (i0 >= a.n) continue;
        auto bisect = [&](int lo, int i) {                       // the last r >= lo with o_r <= i
            int hi = a.R;
            while (hi - lo > 1) {
                const int mid = lo + ((hi - lo) >> 1);
                if (off_at(a, mid) <= i) lo = mid; else hi = mid;
            }
            return lo;
        };
        int r = bisect(0, i0), next = off_at(a, r + 1);
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k;
            if (next <= i && r < a.R - 1) {
                next = off_at(a, ++r + 1);
                if (next <= i) {
                    r = bisect(r, i);
                    next = off_at(a, r + 1);
                }
            }
            v[k] = i >= begin && i < end ? __ldg(a.gE + r) : 0.f;
        }
        *reinterpret_cast<float4*>(a.gat + i0) = make_float4(v[0], v[1], v[2], v[3]);
    }
    double s = 0.0;
    for (int r = blockIdx.x * 256 + threadIdx.x; r < a.R; r += gridDim.x * 256) {
        const int count = off_at(a, r + 1) - off_at(a, r);
        const float g = __ldg(a.gE + r);
        if (count > 0 && g != 0.f) s += (double)g * count;
    }
    __shared__ double ws[8];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
        for (int w = 0; w < 8; ++w) s += ws[w];
        a.part2[blockIdx.x] = s;
    }
}

template <int FW>
__global__ void __launch_bounds__(GRAD_THREADS, 1)
k_readout_grad(const __grid_constant__ CUtensorMap map, ReadoutArgs a)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    // each twice, by the tile's parity
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + GRAD_BAR);
    uint64_t *full = bars, *ready1 = bars + 2, *done1 = bars + 4, *ready2 = bars + 6, *done2 = bars + 8;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 10);
    float* seeds = reinterpret_cast<float*>(sm + GRAD_SEED);
    uint8_t* bytes = sm + GRAD_BYTE;
    uint32_t* gmax = reinterpret_cast<uint32_t*>(sm + GRAD_MAX);
    constexpr int HW = FW / 2, HT = HW / 4;                       // hidden units: all, and a thread's
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int wq = warp & 3, row = wq * 32 + lane;
    const int ntiles = (a.n + 127) / 128;
    const int first = (int)((long long)ntiles * blockIdx.x / a.ncta);
    const int nt = (int)((long long)ntiles * (blockIdx.x + 1) / a.ncta) - first;
    const uint32_t base = smem_u32(sm);
    double* last = reinterpret_cast<double*>(sm + GRAD_X);       // [4][128] column sums, at the end
    auto row0 = [&](int it) { return (first + it) * 128; };
    auto fetch_tile = [&](int it) { tma_tile(base + (it & 1) * TILE_BYTES, &map, row0(it), full + (it & 1)); };

    pdl_trigger();
    StageR1<GRAD_THREADS> r1(a);
    if (warp == 0) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == GRAD_EPI) {                                // the first tiles are on their way before R1 is stored
        for (int k = 0; k < 2; ++k) {
            mbar_init(full + k, 1);
            mbar_init(ready1 + k, 4);
            mbar_init(done1 + k, 1);
            mbar_init(ready2 + k, GRAD_EPI / 32);
            mbar_init(done2 + k, 1);
        }
        fence_mbar_init();
        for (int it = 0; it < 2 && it < nt; ++it) fetch_tile(it);
    }
    float* cst = reinterpret_cast<float*>(sm + GRAD_CST);
    if (threadIdx.x >= 64 && threadIdx.x < 64 + HP)
        cst[threadIdx.x - 64] = (int)threadIdx.x - 64 < a.H ? __ldg(a.c1 + threadIdx.x - 64) * LOG2EF : 0.f;
    const float down = r1.store(sm + GRAD_R1, sm + GRAD_R1 + R1_TERM, reinterpret_cast<uint32_t*>(sm + GRAD_RED));
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);    // D2: 2 x 128 columns, A: 2 x 64, D1: 2 x 64
    const uint32_t tm = tmem + ((uint32_t)(wq * 32) << 16);
    bool ok = true;
    int E = 120, held = 0, cur = 0;                               // the scale, the tiles in D2, and which D2
    // takes note of a tile (x = tile % GRAD_XS): its scale, and whether it goes to the other D2
    // because this one is full or of another scale
    auto plan = [&](uint32_t x) {
        const uint4 m = *reinterpret_cast<const uint4*>(gmax + x * 4);
        const uint32_t mb = max(max(m.x, m.y), max(m.z, m.w));
        const int e = mb >= 0x00800000u ? min(E, max(-120, min(120, 13 - ((int)(mb >> 23) - 127)))) : E;
        const bool other = held >= GRAD_FLUSH || (e < E && held > 0);
        if (other) {
            cur ^= 1;
            held = 0;
        }
        E = e;
        ++held;
        return other;
    };
    // tile `it`'s phase of one of the doubled barriers
    auto wait = [&](uint64_t* two, int it) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(two + (it & 1), (uint32_t)(it >> 1) & 1u, RO_POLLS));
        return ok;
    };
    auto next = [](uint32_t x) { return x == GRAD_XS - 1 ? 0u : x + 1; };

    if (warp >= GRAD_EPI / 32) {
        // ---- widening warps, one row of codes a thread; the first one starts copies and MMAs
        const bool leader = warp == GRAD_EPI / 32;
        const uint32_t go = elect_one();
        const uint32_t id1 = idesc_f16(128, HW, 0, 0), id2 = idesc_f16(128, 2 * HW, 0, 1) | (1u << 15);
        const uint64_t rhi = smem_desc(base + GRAD_R1, HP * 16, 128);
        const uint64_t rlo = smem_desc(base + GRAD_R1 + R1_TERM, HP * 16, 128);
        float seed;                                               // g and scale of this row, of the tile ahead
        int byte;
        auto load = [&](int it) {
            const int i = row0(it) + row;
            const bool in = it < nt && i < a.n;
            seed = in ? a.gat[i] : 0.f;
            byte = in ? (int)__ldg(a.scales + i) : 127;
        };
        auto gemm1 = [&](int it) {
            const uint32_t A = tmem + 256 + (it & 1) * 64, D = tmem + 384 + (it & 1) * 64;
#pragma unroll
            for (int ks = 0; ks < FW / 16; ++ks)                  // the small terms first
                mma_ts(go, D, A + ks * 8, rlo + (uint64_t)((ks * 2 * HP * 16) >> 4), id1, ks > 0 ? 1u : 0u);
#pragma unroll
            for (int ks = 0; ks < FW / 16; ++ks)
                mma_ts(go, D, A + ks * 8, rhi + (uint64_t)((ks * 2 * HP * 16) >> 4), id1, 1u);
            if (go) mma_commit(done1 + (it & 1));
        };
        uint32_t x = 0, xb = 0;                                   // it % GRAD_XS, and the next GEMM2's
        auto gemm2 = [&](int it) {
            plan(xb);
            const uint64_t xd = smem_desc(base + GRAD_X + xb * GRAD_OP, 128, 2048);
            const uint64_t bd = smem_desc(base + GRAD_B + (it & 1) * GRAD_OP, 128, 2048);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)                        // 16 atoms a step
                mma_ss(go, tmem + cur * 128, xd + (uint64_t)((ks * 256) >> 4), bd + (uint64_t)((ks * 256) >> 4), id2,
                       held > 1 || ks > 0 ? 1u : 0u);
            if (go) mma_commit(done2 + (it & 1));
            xb = next(xb);
        };
        pdl_wait();                                               // the seeds
        load(0);
        for (int it = 0; it < nt; ++it) {
            if (!wait(full, it)) break;
            if (it >= 2 && !wait(done1, it - 2)) break;           // A is free
            if (it >= GRAD_XS && !wait(done2, it - GRAD_XS)) break;    // X and the rows' slots are free
            tc_fence_after();                                     // A is overwritten after the MMAs' reads
            const uint32_t src = base + (it & 1) * TILE_BYTES + row * 128;
            const uint32_t to = base + GRAD_X + x * GRAD_OP + row * 16;
#pragma unroll
            for (int q = 0; q < FW / 32; ++q) {
                uint32_t v[16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 w = lds128(src + (((q * 2 + c) ^ (row & 7)) << 4));
                    codes_to_half(w.x, v[c * 8 + 0], v[c * 8 + 1]);
                    codes_to_half(w.y, v[c * 8 + 2], v[c * 8 + 3]);
                    codes_to_half(w.z, v[c * 8 + 4], v[c * 8 + 5]);
                    codes_to_half(w.w, v[c * 8 + 6], v[c * 8 + 7]);
                }
                tmem_st16(tm + 256 + (it & 1) * 64 + q * 16, v);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + (q * 4 + c) * 2048), "r"(v[c * 4]),
                                 "r"(v[c * 4 + 1]), "r"(v[c * 4 + 2]), "r"(v[c * 4 + 3])
                                 : "memory");
            }
            seeds[x * 128 + row] = seed;
            bytes[x * 128 + row] = (uint8_t)byte;
            uint32_t mb = __float_as_uint(seed * __uint_as_float((uint32_t)byte << 23)) & 0x7fffffffu;
            mb = __reduce_max_sync(0xffffffffu, mb >= 0x7f800000u ? 0u : mb);
            if (lane == 0) gmax[x * 4 + wq] = mb;
            load(it + 1);
            fence_proxy_async_smem();
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready1 + (it & 1));
            x = next(x);
            if (leader) {
                if (!wait(ready1, it)) break;
                if (go && it + 2 < nt) fetch_tile(it + 2);        // every row of the stage has been read
                if (it >= 2 && !wait(ready2, it - 2)) break;      // D1 has been read, B written
                tc_fence_after();
                gemm1(it);
                if (it >= 2) gemm2(it - 2);
                __syncwarp();
            }
        }
        if (leader) {
            for (int it = max(nt - 2, 0); it < nt && ok; ++it) {
                if (!wait(ready2, it)) break;
                tc_fence_after();
                gemm2(it);
                __syncwarp();
            }
            if (!ok && go)   // a wait gave up: let the copies and MMAs in flight end (bounded) before the memory goes
                for (int k = 0; k < 10; ++k)
                    for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait_bounded(bars + k, ph, 1u << 12);
        }
    } else {
        // ---- epilogue warps
        const int part = warp >> 2;
        float* sums = a.part + (size_t)blockIdx.x * PART;
        float acc1[HT], acc2[HT];                                 // this thread's columns part * HT + k
        double sum1 = 0.0, sum2 = 0.0;                            // column part * HT + lane % HT, folded
#pragma unroll
        for (int k = 0; k < HT; ++k) acc1[k] = acc2[k] = 0.f;
        int folded = 0;
        bool emptied = false;
        // a D2 of scale 2^e into the CTA's sums (the MMAs that wrote it have completed); an
        // address belongs to one thread, so the order of its additions is fixed
        auto flush = [&](int which, int e) {
            const float un = __uint_as_float((uint32_t)(127 - e) << 23);
            float hi[HT], lo[HT];
            tc_fence_after();
            if (wq * 32 >= FW) return;                            // (features that the narrow form does not have)
            tmem_ld(tm + which * 128 + part * HT, hi);
            tmem_ld(tm + which * 128 + HW + part * HT, lo);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < HT; ++k) {
                float* o = sums + (part * HT + k) * FP + row;
                const float v = (hi[k] - lo[k]) * un;             // the residual is stored negated
                if (emptied) atomicAdd(o, v);
                else *o = v;
            }
            emptied = true;
        };
        auto fold = [&]() {
            sum1 += (double)fold_columns(acc1);
            sum2 += (double)fold_columns(acc2);
#pragma unroll
            for (int k = 0; k < HT; ++k) acc1[k] = acc2[k] = 0.f;
            folded = 0;
        };
        uint32_t x = 0;                                           // it % GRAD_XS
        bool left = false;                                        // the other D2 has to be emptied, of this scale
        int leftE = 0;
        for (int it = 0; it < nt; ++it) {
            if (!wait(done1, it)) break;
            tc_fence_after();
            float d[HT];
            tmem_ld(tm + 384 + (it & 1) * 64 + part * HT, d);
            const bool empty = left;
            const int emptyE = leftE;
            leftE = E;
            left = plan(x);
            if (folded >= GRAD_FOLD) fold();
            // the row's seed, factor and scaled seed; a NaN scale (or weights) makes them NaN,
            // a seed of 0 makes them 0 whatever the row holds
            float gi = seeds[x * 128 + row], k = 0.f, gx = 0.f;
            if (gi != 0.f) {
                const int byte = bytes[x * 128 + row];
                k = row_factor(byte, down);
                if (k != k) gi = k;
                // (half of it: the factor is 2 sigma)
                gx = gi * __uint_as_float((uint32_t)byte << 23) * __uint_as_float((uint32_t)(126 + E) << 23);
            }
            x = next(x);
            if (it >= 2 && !wait(done2, it - 2)) break;           // B is free
            tmem_ld_wait();
            // the D2 that was left at the last tile: its last tile was it - 2.  (Left again at this
            // tile, it is the one that this tile goes to.)
            if (empty) flush(left ? cur : cur ^ 1, emptyE);
            // 8 hidden units, one 16-byte piece of each term, at a time
            const uint32_t to = base + GRAD_B + (it & 1) * GRAD_OP + part * (HT / 8) * 2048 + row * 16;
#pragma unroll
            for (int q = 0; q < HT / 8; ++q) {
                uint32_t h[4], l[4];
                float2 t[4];
                float most = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = q * 8 + 2 * j;
                    const float2 b = *reinterpret_cast<const float2*>(cst + part * HT + c);
                    t[j] = fma2(make_float2(d[c], d[c + 1]), dup2(k), b);
                    t[j] = make_float2(max_nan(t[j].x, -126.f), max_nan(t[j].y, -126.f));
                    most = fmaxf(fmaxf(most, fabsf(t[j].x)), fabsf(t[j].y));
                }
                const bool small = __all_sync(0xffffffffu, most <= SSP2_SMALL);
                float2 y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = q * 8 + 2 * j;
                    y[j] = fma2(dup2(0.5f), make_float2(ex2_mufu(-t[j].x), ex2_mufu(-t[j].y)), dup2(0.5f));
                    const float2 sg = make_float2(rcp_mufu(y[j].x), rcp_mufu(y[j].y));        // 2 sigma
                    const float2 a1 = fma2(dup2(gi), sg, make_float2(acc1[c], acc1[c + 1]));
                    acc1[c] = a1.x; acc1[c + 1] = a1.y;
                    const float2 w = mul2(dup2(gx), sg);
                    split2_neg<0>(w.x, w.y, h[j], l[j]);
                }
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + q * 2048), "r"(h[0]), "r"(h[1]),
                             "r"(h[2]), "r"(h[3])
                             : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + (HW / 8 + q) * 2048), "r"(l[0]), "r"(l[1]),
                             "r"(l[2]), "r"(l[3])
                             : "memory");
                auto sums = [&](auto poly) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = q * 8 + 2 * j;
                        const float2 sp2 = poly ? ssp2_small(t[j])
                                                : add2(t[j], make_float2(lg2_mufu(y[j].x), lg2_mufu(y[j].y)));
                        const float2 a2 = fma2(dup2(gi), sp2, make_float2(acc2[c], acc2[c + 1]));
                        acc2[c] = a2.x; acc2[c + 1] = a2.y;
                    }
                };
                if (small) sums(std::true_type{});
                else sums(std::false_type{});
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready2 + (it & 1));
            ++folded;
        }
        if (ok && nt > 0 && wait(done2, nt - 1)) {
            if (left) flush(cur ^ 1, leftE);
            flush(cur, E);
            fold();
            if (lane < HT) {                                      // (the MMAs have read X)
                last[wq * 128 + part * HT + lane] = sum1;
                last[wq * 128 + 64 + part * HT + lane] = sum2;
            }
        }
    }
    tc_fence_before();
    const int gave_up = __syncthreads_or(!ok);
    if (threadIdx.x < 128) {
        const double* c = last + threadIdx.x;
        a.colpart[(size_t)blockIdx.x * 128 + threadIdx.x] = ((c[0] + c[128]) + c[256]) + c[384];
    } else if (threadIdx.x == 128) {
        a.status[blockIdx.x] = gave_up ? 1u : 0u;
    }
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// dR1 = R2_h sum of the CTAs' D2, dc1 = R2_h / 2 sum of 2 g sigma, dR2 = ln2 sum of g ssp / ln2,
// dc2 = sum_r g_r times the replica's atoms; in float64, in a fixed order.  A CTA takes 32
// columns (CTAs 0 .. 4 H - 1: R1, a quarter of the f of one h each; then 4 for c1 and R2;
// then c2), its 8 warps a share of the partial sums each.
__global__ void __launch_bounds__(256) k_readout_grad_sum(ReadoutArgs a)
{
    pdl_wait();
    __shared__ double red[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, b = blockIdx.x;
    uint32_t bad = (int)threadIdx.x < a.ncta ? a.status[threadIdx.x] : 0u;
    double s = 0.0;
    const int nb = 4 * a.H;
    if (b < nb && (b & 3) * 32 >= a.F) return;                    // inputs that the layer does not have
    if (b < nb) {
        const float* p = a.part + (b >> 2) * FP + (b & 3) * 32 + lane;
#pragma unroll 8
        for (int k = w; k < a.ncta; k += 8) s += (double)p[(size_t)k * PART];
    } else if (b < nb + 4) {
        const double* p = a.colpart + (b - nb) * 32 + lane;
#pragma unroll 8
        for (int k = w; k < a.ncta; k += 8) s += p[(size_t)k * 128];
    }
    red[w][lane] = s;
    bad = __syncthreads_or((int)bad);
    if (w != 0) return;
    s = 0.0;
    for (int k = 0; k < 8; ++k) s += red[k][lane];
    if (b == nb + 4) {                                            // sum_i g_i
        s = 0.0;
        for (int k = lane; k < a.nseed; k += 32) s += a.part2[k];
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    if (bad) s = (double)__int_as_float(0x7fffffff);
    if (b < nb) {
        const int h = b >> 2, f = (b & 3) * 32 + lane;
        if (f < a.F) a.dR1[f * a.H + h] = (float)(s * (double)a.R2[h]);
    } else if (b < nb + 4) {
        const int c = (b - nb) * 32 + lane, h = c & 63;
        if (h < a.H) {
            if (c < 64) a.dc1[h] = (float)(s * 0.5 * (double)a.R2[h]);
            else a.dR2[h] = (float)(s * 0.69314718055994530942);
        }
    } else if (lane == 0) {
        a.dc2[0] = (float)s;
    }
}

// SMs of device dev, asked for once
static int sm_count(int dev)
{
    static std::atomic<int> known[64];
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    n = std::min(n, MAX_SM);
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// more than 48 KB of shared memory for a kernel, once per device
static cudaError_t allow_smem(const void* kernel, uint32_t bytes, int dev, std::atomic<uint64_t>& set)
{
    if (dev < 64 && (set.load() >> dev & 1)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) set.fetch_or((uint64_t)1 << dev);
    return e;
}
static std::atomic<uint64_t> g_fwd_set[2], g_grad_set[2];        // [narrow]

// tensor map of the codes: rows of W bytes, boxes of 128 rows x 128 bytes, 128-byte swizzle
static bool code_map(const ReadoutArgs& a, CUtensorMap* map)
{
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static Encode encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool got = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                         q == cudaDriverEntryPointSuccess;
        return got ? reinterpret_cast<Encode>(p) : nullptr;
    }();
    if (!encode) return false;
    const cuuint64_t dim[2] = {(cuuint64_t)a.W, (cuuint64_t)a.n}, stride[1] = {(cuuint64_t)a.W};
    const cuuint32_t box[2] = {128, 128}, one[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.codes), dim, stride, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static schnet_status readout_args(const uint8_t* codes, const uint8_t* scales, int32_t n, int32_t F, int32_t R,
                                  const int32_t* off, const float* R1, const float* c1, const float* R2, const float* c2,
                                  void* ws, size_t ws_bytes, ReadoutArgs& a)
{
    if (F < 2 || F > FP || (F & 1)) return SCHNET_ERR_UNSUPPORTED;
    size_t need = 0;
    if (n < 0 || n > MAX_ATOMS || R < 1 || R > MAX_REPLICAS || !off || !R1 || !c1 || !R2 || !c2 || !ws ||
        ((uintptr_t)ws & 255) || (n > 0 && (!codes || !scales || ((uintptr_t)codes & 15))) ||
        schnet_readout_workspace_bytes(n, F, &need) != SCHNET_OK || ws_bytes < need)
        return SCHNET_ERR_INVALID_ARG;
    a.codes = codes; a.scales = scales; a.n = n; a.F = F; a.H = F / 2; a.W = (F + 15) / 16 * 16; a.R = R;
    a.off = off; a.R1 = R1; a.c1 = c1; a.R2 = R2; a.c2 = c2;
    return SCHNET_OK;
}

}  // namespace schnet

using namespace schnet;

extern "C" schnet_status schnet_store_features(const void* d_x, int32_t dtype, int64_t n_atoms, int32_t n_features,
                                               int64_t row_stride, uint8_t* d_codes, uint8_t* d_scales,
                                               void* cuda_stream)
{
    if (n_features < 2 || n_features > FP || (n_features & 1)) return SCHNET_ERR_UNSUPPORTED;
    const size_t size = dtype == SCHNET_FLOAT32 ? 4 : 2;
    if (n_atoms < 0 || row_stride < n_features || dtype < SCHNET_FLOAT32 || dtype > SCHNET_BFLOAT16 ||
        (n_atoms > 0 && (!d_x || !d_codes || !d_scales)) || ((uintptr_t)d_codes & 15) || ((uintptr_t)d_x % size))
        return SCHNET_ERR_INVALID_ARG;
    if (cudaPeekAtLastError() != cudaSuccess) return SCHNET_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    cudaError_t e;
    if (dtype == SCHNET_FLOAT32)
        e = store_launch<float>(d_x, n_atoms, n_features, row_stride, nullptr, d_codes, d_scales, s);
    else if (dtype == SCHNET_FLOAT16)
        e = store_launch<__half>(d_x, n_atoms, n_features, row_stride, nullptr, d_codes, d_scales, s);
    else
        e = store_launch<__nv_bfloat16>(d_x, n_atoms, n_features, row_stride, nullptr, d_codes, d_scales, s);
    return e == cudaSuccess ? SCHNET_OK : SCHNET_ERR_CUDA;
}

extern "C" schnet_status schnet_readout_workspace_bytes(int32_t n_atoms, int32_t n_features, size_t* bytes)
{
    if (!bytes || n_atoms < 0 || n_atoms > MAX_ATOMS) return SCHNET_ERR_INVALID_ARG;
    if (n_features < 2 || n_features > FP || (n_features & 1)) return SCHNET_ERR_UNSUPPORTED;
    const size_t tiles = ((size_t)n_atoms + 127) / 128, ctas = std::min<size_t>(tiles, MAX_SM);
    *bytes = sizeof(uint32_t) * MAX_SM +
             std::max(sizeof(double) * 4 * tiles, sizeof(double) * MAX_SEED + ctas * (sizeof(float) * PART + sizeof(double) * 128) +
                                                      sizeof(float) * 128 * tiles);
    return SCHNET_OK;
}

extern "C" schnet_status schnet_readout_energy(const uint8_t* d_codes, const uint8_t* d_scales, int32_t n_atoms,
                                               int32_t n_features, int32_t n_replicas,
                                               const int32_t* d_replica_offsets, const float* d_R1,
                                               const float* d_c1, const float* d_R2, const float* d_c2,
                                               float* d_energy, float* d_eps, void* d_workspace, size_t ws_bytes,
                                               void* cuda_stream)
{
    ReadoutArgs a{};
    schnet_status st = readout_args(d_codes, d_scales, n_atoms, n_features, n_replicas, d_replica_offsets, d_R1,
                                    d_c1, d_R2, d_c2, d_workspace, ws_bytes, a);
    if (st != SCHNET_OK) return st;
    if (!d_energy || (n_atoms > 0 && !d_eps)) return SCHNET_ERR_INVALID_ARG;
    if (cudaPeekAtLastError() != cudaSuccess) return SCHNET_ERR_CUDA;
    a.energy = d_energy;
    a.eps = d_eps;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    int dev = 0;
    if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return enqueued(e);
    a.ncta = std::min((a.n + 127) / 128, sm_count(dev));
    a.status = (uint32_t*)d_workspace;
    a.csum = (double*)(a.status + MAX_SM);
    if (a.n > 0) {
        CUtensorMap map;
        const bool narrow = a.F <= 64;
        const auto f = narrow ? k_readout_eps<64> : k_readout_eps<128>;
        if (!code_map(a, &map)) return SCHNET_ERR_CUDA;
        cudaError_t e = allow_smem((const void*)f, FWD_SMEM, dev, g_fwd_set[narrow]);
        if (e == cudaSuccess) {
            f<<<a.ncta, FWD_THREADS, FWD_SMEM, s>>>(map, a);
            e = cudaPeekAtLastError();
        }
        if (e != cudaSuccess) return enqueued(e);
    }
    return launch_sums(a, s);
}

extern "C" schnet_status schnet_test_readout_timeout(int32_t n_atoms, int32_t n_replicas,
                                                     const int32_t* d_replica_offsets, int32_t given_up,
                                                     float* d_energy, float* d_eps, void* d_workspace,
                                                     size_t ws_bytes, void* cuda_stream)
{
    size_t need = 0;
    if (schnet_readout_workspace_bytes(n_atoms, FP, &need) != SCHNET_OK || n_atoms < 1 || n_replicas < 1 ||
        n_replicas > MAX_REPLICAS || !d_replica_offsets || !d_energy || !d_eps || !d_workspace ||
        ((uintptr_t)d_workspace & 255) || ws_bytes < need)
        return SCHNET_ERR_INVALID_ARG;
    ReadoutArgs a{};
    a.n = n_atoms; a.R = n_replicas; a.off = d_replica_offsets; a.energy = d_energy; a.eps = d_eps;
    a.ncta = std::min((n_atoms + 127) / 128, MAX_SM);
    a.status = (uint32_t*)d_workspace;
    a.csum = (double*)(a.status + MAX_SM);
    cudaStream_t s = (cudaStream_t)cuda_stream;
    cudaError_t e = cudaMemsetAsync(d_workspace, 0, need, s);
    if (e == cudaSuccess && given_up) e = cudaMemsetAsync(a.status + a.ncta - 1, 1, sizeof(uint32_t), s);
    return e == cudaSuccess ? launch_sums(a, s) : enqueued(e);
}

extern "C" schnet_status schnet_readout_gradients(const uint8_t* d_codes, const uint8_t* d_scales, int32_t n_atoms,
                                                  int32_t n_features, int32_t n_replicas,
                                                  const int32_t* d_replica_offsets, const float* d_R1,
                                                  const float* d_c1, const float* d_R2, const float* d_c2,
                                                  const float* d_grad_energy, float* d_dR1, float* d_dc1,
                                                  float* d_dR2, float* d_dc2, void* d_workspace, size_t ws_bytes,
                                                  void* cuda_stream)
{
    ReadoutArgs a{};
    schnet_status st = readout_args(d_codes, d_scales, n_atoms, n_features, n_replicas, d_replica_offsets, d_R1,
                                    d_c1, d_R2, d_c2, d_workspace, ws_bytes, a);
    if (st != SCHNET_OK) return st;
    if (!d_grad_energy || !d_dR1 || !d_dc1 || !d_dR2 || !d_dc2) return SCHNET_ERR_INVALID_ARG;
    if (cudaPeekAtLastError() != cudaSuccess) return SCHNET_ERR_CUDA;
    a.gE = d_grad_energy;
    a.dR1 = d_dR1; a.dc1 = d_dc1; a.dR2 = d_dR2; a.dc2 = d_dc2;
    int dev = 0;
    if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return enqueued(e);
    a.ncta = std::min((a.n + 127) / 128, sm_count(dev));
    a.status = (uint32_t*)d_workspace;
    a.nseed = a.n > 0 ? std::min(std::max((a.n + SEED_ATOMS - 1) / SEED_ATOMS, (a.R + 1023) / 1024), MAX_SEED) : 0;
    a.part2 = (double*)(a.status + MAX_SM);
    a.colpart = a.part2 + MAX_SEED;
    a.part = (float*)(a.colpart + (size_t)a.ncta * 128);
    a.gat = a.part + (size_t)a.ncta * PART;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    if (a.n > 0) {
        CUtensorMap map;
        const bool narrow = a.F <= 64;
        const auto f = narrow ? k_readout_grad<64> : k_readout_grad<128>;
        if (!code_map(a, &map)) return SCHNET_ERR_CUDA;
        cudaError_t e = allow_smem((const void*)f, GRAD_SMEM, dev, g_grad_set[narrow]);
        if (e == cudaSuccess) {
            k_readout_seeds<<<a.nseed, 256, 0, s>>>(a);
            e = cudaPeekAtLastError();
        }
        if (e == cudaSuccess) e = launch_pdl(f, a.ncta, GRAD_THREADS, GRAD_SMEM, s, map, a);
        if (e != cudaSuccess) return enqueued(e);
    }
    return enqueued(launch_pdl(k_readout_grad_sum, 4 * a.H + 5, 256, 0, s, a));
}
