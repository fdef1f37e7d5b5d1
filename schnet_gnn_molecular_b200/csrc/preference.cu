// Preference loss over pairs of conformations: forward and gradient in one pass
// over the pairs (no counterpart on the pages).
//
// Under p(x) ~ exp(-E(x)/kT), ln p_w - ln p_l = -(E_w - E_l)/kT: the partition
// function cancels.  m = -[(E_w - Eref_w) - (E_l - Eref_l)]/kT; a pair's loss is
// (1-s) ln(1+e^-m) + s ln(1+e^m), its slope c = dL/dm = sigma(m) - (1-s), |c| <= 1.
// The gradient scatters -c to w and +c to l.  A replica may be in any number of pairs,
// so the scatter is an atomic sum; it is made of 64-bit integers, whose sum does not
// depend on the order, so the gradient is the same bits every run:
//   word 0: c in units of 2^-s0, s0 = 62 - b, b = bits of n_pairs (|sum| < 2^62);
//   word 1: the slopes below 2^(24-s0), which word 0 would keep to less than 2^-25
//           of themselves, in units of 2^-s1, s1 = 2 s0 - 24 (|sum| < 2^62 again).
// A pair's slope goes to one of the two words, so there are two atomics a pair.
// A pass over the pairs is bound by its scattered accesses' way out of the SM, a sector each:
// 2 gathers (the energies' gaps E - Eref are formed first) and 2 atomics.  4 M pairs among 1 M
// replicas: the port from L1 to the crossbar is 81 % busy (HBM 8 %, L2's tags 29 %); the call
// takes 109 us with both energies gathered, 82 us so.
#include <algorithm>
#include <cmath>

#include "internal.h"

namespace schnet {

constexpr int PT = 256;                  // threads per CTA
constexpr int PREF_MAX_CTA = 148 * 8;
constexpr int PREF_N = 4;                // pairs a thread has in flight

struct PrefPartial {
    double loss;
    long long count;
    unsigned int flags, pad;
};

struct PrefArgs {
    const void *energy, *reference;
    const int2* pairs;
    long long P;
    int R;
    double inv_kT, s;
    int s0, s1;
    double* loss;
    float *margins, *grad;
    uint32_t* flags;
    double* gap;                         // [R] E - Eref
    unsigned long long *w0, *w1;         // [R] slope sums
    unsigned char* bad;                  // [R] 1: a NaN margin touches the replica
    PrefPartial* partial;                // [CTAs of the pair pass]
};

// whether a pair counts
__device__ __forceinline__ bool pair_ok(const PrefArgs& a, int2 q, unsigned int& flags)
{
    if ((unsigned)q.x < (unsigned)a.R && (unsigned)q.y < (unsigned)a.R) return true;
    if (q.x < -1 || q.x >= a.R || q.y < -1 || q.y >= a.R) flags |= SCHNET_FLAG_BADINDEX;
    return false;
}

// replica r's energy above the reference
template <class T>
__device__ __forceinline__ double gap_of(const PrefArgs& a, int r)
{
    const double e = (double)__ldg(static_cast<const T*>(a.energy) + r);
    return a.reference ? e - (double)__ldg(static_cast<const T*>(a.reference) + r) : e;
}

// loss and slope of a margin: t = e^-|m|, ln(1+e^-|m|) = log1p(t), and the logistic of
// the sign that does not cancel
__device__ __forceinline__ void pair_loss(double m, double s, double& loss, double& c)
{
    const double t = exp(-fabs(m));
    const double r = 1.0 / (1.0 + t);
    loss = log1p(t);
    if (m < 0.0 && s < 1.0) loss -= (1.0 - s) * m;
    if (m > 0.0 && s > 0.0) loss += s * m;         // (an infinite margin times a weight of 0 is 0)
    if (isnan(m)) loss = m;
    const double sneg = m >= 0.0 ? t * r : r;      // sigma(-m)
    c = s - sneg;                                  // = sigma(m) - (1 - s), no cancellation at s = 0
}

// The units of the two words, and the border between them.
struct Units {
    double u0, u1, border;
    __device__ explicit Units(const PrefArgs& a) : u0(power(a.s0)), u1(power(a.s1)), border(power(24 - a.s0)) {}
    static __device__ double power(int e) { return __longlong_as_double((long long)(1023 + e) << 52); }
};

// N pairs, `step` apart: margins out, slopes into the words, loss and count to the thread's
// sums.  All of them are loaded, then all their energies, before the first is worked on:
// the gathers' latency is what a thread waits for.
template <int N>
__device__ __forceinline__ void some_pairs(const PrefArgs& a, const Units& u, long long p, long long step,
                                           const double* gap, unsigned long long* w0, unsigned long long* w1, unsigned char* bad,
                                           double& loss, long long& count, unsigned int& flags)
{
    int2 q[N];
    double m[N];
    bool ok[N];
#pragma unroll
    for (int k = 0; k < N; ++k) q[k] = p + k * step < a.P ? __ldg(a.pairs + p + k * step) : make_int2(-1, -1);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        ok[k] = pair_ok(a, q[k], flags);
        m[k] = ok[k] ? (gap[q[k].y] - gap[q[k].x]) * a.inv_kT : 0.0;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (a.margins && p + k * step < a.P) a.margins[p + k * step] = (float)m[k];
        if (!ok[k]) continue;
        double l, c;
        pair_loss(m[k], a.s, l, c);
        loss += l;
        count += 1;
        if (isnan(m[k])) {
            flags |= SCHNET_FLAG_NONFINITE;
            bad[q[k].x] = 1;
            bad[q[k].y] = 1;
            continue;
        }
        const bool fine = fabs(c) < u.border;
        const long long v = __double2ll_rn(c * (fine ? u.u1 : u.u0));
        unsigned long long* w = fine ? w1 : w0;
        if (v != 0 && q[k].x != q[k].y) {
            atomicAdd(w + q[k].x, (unsigned long long)(-v));
            atomicAdd(w + q[k].y, (unsigned long long)v);
        }
    }
}

__device__ __forceinline__ float slope_of(const PrefArgs& a, double scale, unsigned long long w0, unsigned long long w1,
                                          unsigned char bad)
{
    if (bad) return __int_as_float(0x7fffffff);
    return (float)(((double)(long long)w0 * Units::power(-a.s0) + (double)(long long)w1 * Units::power(-a.s1)) * scale);
}

// the CTA's sums in a fixed order, valid in thread 0
template <int THREADS>
__device__ __forceinline__ PrefPartial cta_sums(double loss, long long count, unsigned int flags)
{
    __shared__ PrefPartial part[THREADS / 32];
    for (int o = 16; o > 0; o >>= 1) {
        loss += __shfl_xor_sync(0xffffffffu, loss, o);
        count += __shfl_xor_sync(0xffffffffu, count, o);
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = PrefPartial{loss, count, flags, 0u};
    __syncthreads();
    PrefPartial t{0.0, 0, 0u, 0u};
    if (threadIdx.x == 0)
        for (int w = 0; w < THREADS / 32; ++w) {
            t.loss += part[w].loss;
            t.count += part[w].count;
            t.flags |= part[w].flags;
        }
    return t;
}

template <class T>
__global__ void __launch_bounds__(PT) k_pref_gaps(PrefArgs a)
{
    pdl_trigger();
    for (int r = blockIdx.x * PT + threadIdx.x; r < a.R; r += gridDim.x * PT) {
        a.gap[r] = gap_of<T>(a, r);
        a.w0[r] = a.w1[r] = 0;
        a.bad[r] = 0;
    }
}

__global__ void __launch_bounds__(PT) k_pref_pairs(PrefArgs a)
{
    pdl_trigger();
    pdl_wait();
    double loss = 0.0;
    long long count = 0;
    unsigned int flags = 0;
    const Units u(a);
    const long long step = (long long)gridDim.x * PT;
    for (long long p = (long long)blockIdx.x * PT + threadIdx.x; p < a.P; p += step * PREF_N)
        some_pairs<PREF_N>(a, u, p, step, a.gap, a.w0, a.w1, a.bad, loss, count, flags);
    const PrefPartial t = cta_sums<PT>(loss, count, flags);
    if (threadIdx.x == 0) a.partial[blockIdx.x] = t;
}

// Everything in one CTA, the words in shared memory, where pairs and replicas are few: one
// launch instead of three.  A call takes (queued / on the device, us) 6.2 / 4.3 with 512 pairs
// and 8.2 / 6.0 with 1024, against 10.5 / 5.2 and 10.5 / 4.7 in three; 2048 pairs, whose
// float64 logarithms one SM works on alone, 10.3 / 9.1 against 10.5 / 4.7.
constexpr int SMALL_T = 512, SMALL_P = 1024, SMALL_R = 1792;       // 42 KB + 1.8 KB of shared memory at most
template <class T>
__global__ void __launch_bounds__(SMALL_T) k_pref_small(PrefArgs a)
{
    extern __shared__ double small_gap[];                     // [R], then the words
    unsigned long long *w0 = reinterpret_cast<unsigned long long*>(small_gap + a.R), *w1 = w0 + a.R;
    __shared__ unsigned char bad[SMALL_R];
    __shared__ PrefPartial total;
    for (int r = threadIdx.x; r < a.R; r += SMALL_T) {
        small_gap[r] = gap_of<T>(a, r);
        w0[r] = w1[r] = 0;
        bad[r] = 0;
    }
    __syncthreads();
    double loss = 0.0;
    long long count = 0;
    unsigned int flags = 0;
    const Units u(a);
    for (long long p = threadIdx.x; p < a.P; p += SMALL_T * 2)
        some_pairs<2>(a, u, p, SMALL_T, small_gap, w0, w1, bad, loss, count, flags);
    const PrefPartial t = cta_sums<SMALL_T>(loss, count, flags);
    if (threadIdx.x == 0) total = t;
    __syncthreads();
    const double inv = total.count > 0 ? 1.0 / (double)total.count : 0.0;
    if (threadIdx.x == 0) {
        *a.loss = total.loss * inv;
        if (a.flags) *a.flags = total.flags;
    }
    for (int r = threadIdx.x; r < a.R; r += SMALL_T) a.grad[r] = slope_of(a, a.inv_kT * inv, w0[r], w1[r], bad[r]);
}

__global__ void __launch_bounds__(PT) k_pref_finish(PrefArgs a, int nparts)
{
    pdl_wait();
    __shared__ PrefPartial total;
    double loss = 0.0;
    long long count = 0;
    unsigned int flags = 0;
    for (int k = threadIdx.x; k < nparts; k += PT) {
        const PrefPartial t = a.partial[k];
        loss += t.loss;
        count += t.count;
        flags |= t.flags;
    }
    const PrefPartial t = cta_sums<PT>(loss, count, flags);
    if (threadIdx.x == 0) total = t;
    __syncthreads();
    const double inv = total.count > 0 ? 1.0 / (double)total.count : 0.0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.loss = total.loss * inv;
        if (a.flags) *a.flags = total.flags;
    }
    for (int r = blockIdx.x * PT + threadIdx.x; r < a.R; r += gridDim.x * PT)
        a.grad[r] = slope_of(a, a.inv_kT * inv, a.w0[r], a.w1[r], a.bad[r]);
}

static size_t pref_carve(int R, uint8_t* base, PrefArgs& a)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    size_t off = 0;
    a.gap = reinterpret_cast<double*>(base + off);
    off += up((size_t)R * 8);
    a.w0 = reinterpret_cast<unsigned long long*>(base + off);
    off += up((size_t)R * 8);
    a.w1 = reinterpret_cast<unsigned long long*>(base + off);
    off += up((size_t)R * 8);
    a.bad = base + off;
    off += up((size_t)R);
    a.partial = reinterpret_cast<PrefPartial*>(base + off);
    off += up(sizeof(PrefPartial) * PREF_MAX_CTA);
    return off;
}

}  // namespace schnet

using namespace schnet;

extern "C" schnet_status schnet_preference_workspace_bytes(int32_t n_replicas, int64_t n_pairs, size_t* bytes)
{
    if (!bytes || n_replicas < 1 || n_replicas > MAX_REPLICAS || n_pairs < 0 || n_pairs > 0x7fffffffLL)
        return SCHNET_ERR_INVALID_ARG;
    PrefArgs a{};
    *bytes = pref_carve(n_replicas, nullptr, a);
    return SCHNET_OK;
}

extern "C" schnet_status schnet_preference_loss(const void* d_energy, const void* d_reference, int32_t dtype,
                                                int32_t n_replicas, const int32_t* d_pairs, int64_t n_pairs,
                                                double kT, double smoothing, double* d_loss, float* d_margins,
                                                float* d_grad_energy, uint32_t* d_flags, void* d_workspace,
                                                size_t ws_bytes, void* cuda_stream)
{
    size_t need = 0;
    if (!d_energy || !d_loss || !d_grad_energy || !d_workspace || ((uintptr_t)d_workspace & 255) ||
        (dtype != SCHNET_FLOAT32 && dtype != SCHNET_FLOAT64) || !(kT > 0.0) || !std::isfinite(kT) ||
        !std::isfinite(1.0 / kT) || !(smoothing >= 0.0 && smoothing <= 1.0) ||
        schnet_preference_workspace_bytes(n_replicas, n_pairs, &need) != SCHNET_OK || ws_bytes < need ||
        (n_pairs > 0 && !d_pairs) || ((uintptr_t)d_pairs & 7))
        return SCHNET_ERR_INVALID_ARG;
    if (cudaPeekAtLastError() != cudaSuccess) return SCHNET_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    PrefArgs a{};
    pref_carve(n_replicas, (uint8_t*)d_workspace, a);
    a.energy = d_energy;
    a.reference = d_reference;
    a.pairs = reinterpret_cast<const int2*>(d_pairs);
    a.P = n_pairs;
    a.R = n_replicas;
    a.inv_kT = 1.0 / kT;
    a.s = smoothing;
    int b = 0;
    while ((n_pairs >> b) > 0) ++b;
    a.s0 = 62 - b;
    a.s1 = 2 * a.s0 - 24;
    a.loss = d_loss;
    a.margins = d_margins;
    a.grad = d_grad_energy;
    a.flags = d_flags;
    const bool f64 = dtype == SCHNET_FLOAT64;
    if (n_pairs <= SMALL_P && n_replicas <= SMALL_R) {
        const size_t smem = (size_t)n_replicas * 24;
        if (f64) k_pref_small<double><<<1, SMALL_T, smem, s>>>(a);
        else k_pref_small<float><<<1, SMALL_T, smem, s>>>(a);
        return enqueued(cudaSuccess);
    }
    const int g1 = (int)std::max<int64_t>(1, std::min<int64_t>((n_pairs + PT - 1) / PT, PREF_MAX_CTA));
    const int g2 = std::min((n_replicas + PT - 1) / PT, PREF_MAX_CTA);
    if (f64) k_pref_gaps<double><<<g2, PT, 0, s>>>(a);
    else k_pref_gaps<float><<<g2, PT, 0, s>>>(a);
    cudaError_t e = cudaPeekAtLastError();
    if (e == cudaSuccess) e = launch_pdl(k_pref_pairs, g1, PT, 0, s, a);
    if (e == cudaSuccess) e = launch_pdl(k_pref_finish, g2, PT, 0, s, a, g1);
    return enqueued(e);
}
