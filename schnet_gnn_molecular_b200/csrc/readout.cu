// Readout tuning from stored features: the 8-bit store, readout energies and the
// readout's weight gradients (no counterpart on the pages; the readout is the model's
// eps = ssp(x R1 + c1) R2 + c2, hidden width H = F/2).
//
// Store: per row (at most 128 features, one block) the scale is a power of two, so
// x / scale is exact and the e4m3 rounding is the only one: codes are a function of
// x alone, whatever computes them.
#include <algorithm>

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
constexpr int RT = 256;                  // threads per CTA
constexpr int RTILE = 32;                // atoms a CTA stages at a time

struct ReadoutArgs {
    const uint8_t *codes, *scales;
    int n, F, H, W, R;
    const int32_t* off;
    const float *R1, *c1, *R2, *c2;
    float *energy, *eps;
    const float* gE;
    float *dR1, *dc1, *dR2, *dc2;
    float* part;                         // [CTAs][F H + 2 H] partial gradients
    double* part2;                       // [CTAs] partial dc2
};

__device__ __forceinline__ int off_at(const ReadoutArgs& a, int r) { return min(max(__ldg(a.off + r), 0), a.n); }

// the replica of atom i, -1 for none: the last r with o_r <= i, if i < o_{r+1}
__device__ __forceinline__ int replica_of(const ReadoutArgs& a, int i)
{
    if (i < off_at(a, 0) || i >= off_at(a, a.R)) return -1;
    int lo = 0, hi = a.R - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off_at(a, mid) <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// stage x_i (stored values) of the tile's atoms as [RTILE][F]
__device__ __forceinline__ void stage_features(const ReadoutArgs& a, int i0, float* xs)
{
    for (int k = threadIdx.x; k < RTILE * a.F; k += RT) {
        const int i = i0 + k / a.F, f = k % a.F;
        float v = 0.f;
        if (i < a.n) {
            const int b = a.scales[i];
            const __half_raw h = __nv_cvt_fp8_to_halfraw(a.codes[(size_t)i * a.W + f], __NV_E4M3);
            v = b == 255 ? __int_as_float(0x7fffffff) : __half2float(__half(h)) * __uint_as_float((uint32_t)b << 23);
        }
        xs[k] = v;
    }
}

__global__ void __launch_bounds__(RT) k_readout_eps(ReadoutArgs a)
{
    extern __shared__ float rsm[];
    float* xs = rsm;                     // [RTILE][F]
    float* w = rsm + RTILE * a.F;        // [F][H]
    for (int k = threadIdx.x; k < a.F * a.H; k += RT) w[k] = a.R1[k];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float c2 = a.c2[0];
    for (int i0 = blockIdx.x * RTILE; i0 < a.n; i0 += gridDim.x * RTILE) {
        __syncthreads();
        stage_features(a, i0, xs);
        __syncthreads();
        for (int k = warp; k < RTILE && i0 + k < a.n; k += RT / 32) {
            float e = 0.f;
            for (int h = lane; h < a.H; h += 32) {
                float p = a.c1[h];
                for (int f = 0; f < a.F; ++f) p = fmaf(xs[k * a.F + f], w[f * a.H + h], p);
                e = fmaf(ssp(p), a.R2[h], e);
            }
            for (int o = 16; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
            if (lane == 0) a.eps[i0 + k] = e + c2;
        }
    }
}

__global__ void __launch_bounds__(RT) k_readout_sums(ReadoutArgs a)
{
    const int r = blockIdx.x;
    double s = 0.0;
    const int hi = off_at(a, r + 1);
    for (int i = off_at(a, r) + threadIdx.x; i < hi; i += RT) s += (double)a.eps[i];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __shared__ double ws[RT / 32];
    if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < RT / 32; ++w) t += ws[w];
        a.energy[r] = (float)t;
    }
}

// ---------------------------------------------------------------------------
// readout weight gradients
// ---------------------------------------------------------------------------
constexpr int GRAD_CTA = 148;

// Tile by tile: stage x, form the hidden layer again, stage dp and g ssp(p), then every
// thread adds its entries of x^T dp.  One partial per CTA, summed in a fixed order.
__global__ void __launch_bounds__(RT) k_readout_grad(ReadoutArgs a)
{
    extern __shared__ float rsm[];
    float* xs = rsm;                               // [RTILE][F]
    float* w = xs + RTILE * a.F;                   // [F][H]
    float* dp = w + a.F * a.H;                     // [RTILE][H]
    float* ga = dp + RTILE * a.H;                  // [RTILE][H]
    __shared__ float g[RTILE];
    for (int k = threadIdx.x; k < a.F * a.H; k += RT) w[k] = a.R1[k];
    constexpr int MAXE = FP * HP / RT;
    float acc[MAXE], col = 0.f;
#pragma unroll
    for (int k = 0; k < MAXE; ++k) acc[k] = 0.f;
    double gsum = 0.0;
    for (int i0 = blockIdx.x * RTILE; i0 < a.n; i0 += gridDim.x * RTILE) {
        __syncthreads();
        stage_features(a, i0, xs);
        if (threadIdx.x < RTILE) {
            const int i = i0 + threadIdx.x;
            const int r = i < a.n ? replica_of(a, i) : -1;
            g[threadIdx.x] = r >= 0 ? a.gE[r] : 0.f;
            gsum += (double)g[threadIdx.x];
        }
        __syncthreads();
        for (int k = threadIdx.x; k < RTILE * a.H; k += RT) {
            const int i = k / a.H, h = k % a.H;
            float p = a.c1[h];
            for (int f = 0; f < a.F; ++f) p = fmaf(xs[i * a.F + f], w[f * a.H + h], p);
            const bool in = g[i] != 0.f;           // an atom of no replica adds nothing, whatever it holds
            dp[k] = in ? g[i] * a.R2[h] * sigmoidf(p) : 0.f;
            ga[k] = in ? g[i] * ssp(p) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < MAXE; ++k) {
            const int e = threadIdx.x + k * RT;
            if (e < a.F * a.H) {
                const int f = e / a.H, h = e % a.H;
                for (int i = 0; i < RTILE; ++i)
                    if (g[i] != 0.f) acc[k] = fmaf(xs[i * a.F + f], dp[i * a.H + h], acc[k]);
            }
        }
        if (threadIdx.x < 2 * a.H) {
            const int h = threadIdx.x % a.H;
            const float* src = threadIdx.x < a.H ? dp : ga;
            for (int i = 0; i < RTILE; ++i) col += src[i * a.H + h];
        }
    }
    float* out = a.part + (size_t)blockIdx.x * (a.F * a.H + 2 * a.H);
#pragma unroll
    for (int k = 0; k < MAXE; ++k) {
        const int e = threadIdx.x + k * RT;
        if (e < a.F * a.H) out[e] = acc[k];
    }
    if (threadIdx.x < 2 * a.H) out[a.F * a.H + threadIdx.x] = col;
    if (threadIdx.x < 32) {
        for (int o = 16; o > 0; o >>= 1) gsum += __shfl_xor_sync(0xffffffffu, gsum, o);
        if (threadIdx.x == 0) a.part2[blockIdx.x] = gsum;
    }
}

__global__ void __launch_bounds__(RT) k_readout_grad_sum(ReadoutArgs a, int nparts)
{
    const int fh = a.F * a.H, m = fh + 2 * a.H;
    const int k = blockIdx.x * RT + threadIdx.x;
    if (k < m) {
        double s = 0.0;
        for (int c = 0; c < nparts; ++c) s += (double)a.part[(size_t)c * m + k];
        if (k < fh) a.dR1[k] = (float)s;
        else if (k < fh + a.H) a.dc1[k - fh] = (float)s;
        else a.dR2[k - fh - a.H] = (float)s;
    } else if (k == m) {
        double s = 0.0;
        for (int c = 0; c < nparts; ++c) s += a.part2[c];
        a.dc2[0] = (float)s;
    }
}

static schnet_status readout_args(const uint8_t* codes, const uint8_t* scales, int32_t n, int32_t F, int32_t R,
                                  const int32_t* off, const schnet_readout* w, void* ws, size_t ws_bytes,
                                  ReadoutArgs& a)
{
    if (F < 2 || F > FP || (F & 1)) return SCHNET_ERR_UNSUPPORTED;
    size_t need = 0;
    if (n < 0 || R < 1 || !off || !w || !w->R1 || !w->c1 || !w->R2 || !w->c2 || !ws || ((uintptr_t)ws & 255) ||
        (n > 0 && (!codes || !scales || ((uintptr_t)codes & 15))) ||
        schnet_readout_workspace_bytes(n, F, &need) != SCHNET_OK || ws_bytes < need)
        return SCHNET_ERR_INVALID_ARG;
    a.codes = codes; a.scales = scales; a.n = n; a.F = F; a.H = F / 2; a.W = (F + 15) / 16 * 16; a.R = R;
    a.off = off; a.R1 = w->R1; a.c1 = w->c1; a.R2 = w->R2; a.c2 = w->c2;
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
    if (!bytes || n_atoms < 0) return SCHNET_ERR_INVALID_ARG;
    if (n_features < 2 || n_features > FP || (n_features & 1)) return SCHNET_ERR_UNSUPPORTED;
    const size_t H = n_features / 2;
    *bytes = GRAD_CTA * (sizeof(double) + sizeof(float) * (n_features * H + 2 * H)) + 512;
    return SCHNET_OK;
}

extern "C" schnet_status schnet_readout_energy(const uint8_t* d_codes, const uint8_t* d_scales, int32_t n_atoms,
                                               int32_t n_features, int32_t n_replicas,
                                               const int32_t* d_replica_offsets, const schnet_readout* w,
                                               float* d_energy, float* d_eps, void* d_workspace, size_t ws_bytes,
                                               void* cuda_stream)
{
    ReadoutArgs a{};
    schnet_status st = readout_args(d_codes, d_scales, n_atoms, n_features, n_replicas, d_replica_offsets, w,
                                    d_workspace, ws_bytes, a);
    if (st != SCHNET_OK) return st;
    if (!d_energy || (n_atoms > 0 && !d_eps)) return SCHNET_ERR_INVALID_ARG;
    if (cudaPeekAtLastError() != cudaSuccess) return SCHNET_ERR_CUDA;
    a.energy = d_energy;
    a.eps = d_eps;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    const size_t smem = sizeof(float) * (RTILE * a.F + a.F * a.H);
    if (cudaFuncSetAttribute(k_readout_eps, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return SCHNET_ERR_CUDA;
    if (a.n > 0) k_readout_eps<<<std::min((a.n + RTILE - 1) / RTILE, 148 * 4), RT, smem, s>>>(a);
    k_readout_sums<<<a.R, RT, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SCHNET_OK : SCHNET_ERR_CUDA;
}

extern "C" schnet_status schnet_readout_gradients(const uint8_t* d_codes, const uint8_t* d_scales, int32_t n_atoms,
                                                  int32_t n_features, int32_t n_replicas,
                                                  const int32_t* d_replica_offsets, const schnet_readout* w,
                                                  const float* d_grad_energy, float* d_dR1, float* d_dc1,
                                                  float* d_dR2, float* d_dc2, void* d_workspace, size_t ws_bytes,
                                                  void* cuda_stream)
{
    ReadoutArgs a{};
    schnet_status st = readout_args(d_codes, d_scales, n_atoms, n_features, n_replicas, d_replica_offsets, w,
                                    d_workspace, ws_bytes, a);
    if (st != SCHNET_OK) return st;
    if (!d_grad_energy || !d_dR1 || !d_dc1 || !d_dR2 || !d_dc2) return SCHNET_ERR_INVALID_ARG;
    if (cudaPeekAtLastError() != cudaSuccess) return SCHNET_ERR_CUDA;
    a.gE = d_grad_energy;
    a.dR1 = d_dR1; a.dc1 = d_dc1; a.dR2 = d_dR2; a.dc2 = d_dc2;
    a.part2 = (double*)d_workspace;
    a.part = (float*)(a.part2 + GRAD_CTA);
    cudaStream_t s = (cudaStream_t)cuda_stream;
    const size_t smem = sizeof(float) * (RTILE * a.F + a.F * a.H + 2 * RTILE * a.H);
    if (cudaFuncSetAttribute(k_readout_grad, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return SCHNET_ERR_CUDA;
    const int grid = std::max(1, std::min((a.n + RTILE - 1) / RTILE, GRAD_CTA));
    k_readout_grad<<<grid, RT, smem, s>>>(a);
    k_readout_grad_sum<<<(a.F * a.H + 2 * a.H + RT) / RT, RT, 0, s>>>(a, grid);
    return cudaGetLastError() == cudaSuccess ? SCHNET_OK : SCHNET_ERR_CUDA;
}
