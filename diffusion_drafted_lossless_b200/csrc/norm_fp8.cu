// norm_fp8.cu — RMS norm with the residual's addition and e4m3 output, and the e4m3
// quantiser of weights and activations.
//
//   h = x + residual,  u = h * weight,  rstd = 1 / sqrt(mean h^2 + eps),  y = u rstd
//   per block, a = max |u|:  scale = max(a rstd / 448, 2^-126),  value = e4m3(448 u / a)
// The row's factor rstd cancels in the values, so they need no statistics: only the scales
// do. The quotient 448 u / a is what is rounded, once, to nearest even:
//   bf16 inputs: u is exact in float32 (a product of two 8-bit significands), and 448 / a is
//     taken as a float32 and its float32 remainder, so that the quotient carries 2^-24 of
//     relative error. 448 u and border * a are whole numbers of at most 21 bits on a common
//     scale, so a quotient that is not on a border of e4m3 is at least 2^-21 away from it
//     and one that is on it comes out exactly: the values are those of exact arithmetic.
//   float32 inputs: the same in float64 (u is exact there), rounded to float32 to odd so
//     that the second rounding, to e4m3, sees on which side of a border the quotient lies.
//
// Bound: HBM. The norm reads x and the residual and writes h, the values and, if asked, y,
// each once; a row is held in shared memory between its sum of squares and its values (16
// bytes a thread at a time, read back by the thread that wrote them). One CTA per row.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "layers.cuh"

namespace uno {

int device_sms() {
    static std::atomic<int> cache[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

namespace {

// 16 bytes of a row: 8 bf16 or 4 float32 values
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);
// lanes that hold one 128-column block
template <typename T>
constexpr int kLanes = kBlockCols / kVec<T>;

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[kVec<T>]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (std::is_same_v<T, float>) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[kVec<T>]) {
    if constexpr (std::is_same_v<T, float>)
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else
        return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// the arithmetic a block's values are found in
template <typename T>
using Wide = std::conditional_t<std::is_same_v<T, float>, double, float>;

template <typename U>
__device__ __forceinline__ U group_max(U v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) {
            const U w = __shfl_xor_sync(kFullMask, v, o);
            v = w > v ? w : v;
        }
    return v;
}

// float64 to float32, to odd: a value between two float32 numbers goes to the one whose last
// bit is set, so rounding the result again to a much shorter type rounds the value itself
__device__ __forceinline__ float to_odd(double t) {
    const uint32_t inexact = (__double2loint(t) & 0x1FFFFFFF) != 0 ? 1u : 0u;
    return __uint_as_float(__float_as_uint(__double2float_rz(t)) | inexact);
}

// The quotients of a block's 16-byte piece u by its scale, and the scale. a: the block's
// largest |u|. factor: the row's rstd (1 for the quantiser).
template <typename T>
__device__ __forceinline__ float block_quotients(const Wide<T> (&u)[kVec<T>], Wide<T> a, float factor,
                                                 float (&t)[kVec<T>]) {
    float scale = std::is_same_v<T, float> ? (float)((double)a * (double)factor / 448.0)
                                           : __fdiv_rn((float)a * factor, kE4m3Max);
    if constexpr (!std::is_same_v<T, float>) {
        // far from overflow and underflow of 448 / a and its remainder
        if (a >= 0x1p-90f && a <= 0x1p90f && scale >= kMinScale) {
            const float c = __fdiv_rn(kE4m3Max, a);
            const float r = __fdiv_rn(fmaf(-c, a, kE4m3Max), a);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) t[i] = fmaf(u[i], c, u[i] * r);
            return scale;
        }
    }
    double top = (double)a;
    if (scale < kMinScale) {
        scale = kMinScale;
        const double least = 448.0 * (double)kMinScale / (double)factor;
        top = top > least ? top : least;
    }
    const double c = 448.0 / top, r = fma(-c, top, 448.0) / top;
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) t[i] = to_odd(fma((double)u[i], c, (double)u[i] * r));
    return scale;
}

// kVec<T> e4m3 values to out
template <typename T>
__device__ __forceinline__ void store_values(uint8_t* out, const float (&t)[kVec<T>]) {
    if constexpr (std::is_same_v<T, float>)
        *reinterpret_cast<uint32_t*>(out) = e4m3x4(t[0], t[1], t[2], t[3]);
    else
        *reinterpret_cast<uint2*>(out) = make_uint2(e4m3x4(t[0], t[1], t[2], t[3]), e4m3x4(t[4], t[5], t[6], t[7]));
}

template <typename T>
__device__ __forceinline__ Wide<T> piece_max(const Wide<T> (&u)[kVec<T>]) {
    Wide<T> a = 0;
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) a = fmax(a, fabs(u[i]));  // (a NaN is passed over)
    return a;
}

constexpr int kNormThreads = 512;

// (x and residual may be out_residual: no restrict, no read-only loads. A thread reads its
// 16 bytes before it writes them.)
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const T* x, const T* residual, const T* __restrict__ weight,
                                                            int d, float eps, T* out_residual,
                                                            uint8_t* __restrict__ out_q, float* __restrict__ out_scale,
                                                            T* __restrict__ out_y) {
    extern __shared__ uint4 row_h[];
    __shared__ float part[kNormThreads / 32];
    constexpr int V = kVec<T>;
    const int nvec = d / V, nt = blockDim.x, lane = threadIdx.x & 31;
    const int64_t at = (int64_t)blockIdx.x * d;
    float ss = 0.f;
    for (int c = threadIdx.x; c < nvec; c += nt) {
        uint4 v = *reinterpret_cast<const uint4*>(x + at + (int64_t)c * V);
        float h[V];
        unpack<T>(v, h);
        if (residual) {
            float r[V];
            unpack<T>(*reinterpret_cast<const uint4*>(residual + at + (int64_t)c * V), r);
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] += r[i];
            v = pack<T>(h);
            unpack<T>(v, h);  // the rounded sum is what is normed
            if (out_residual) *reinterpret_cast<uint4*>(out_residual + at + (int64_t)c * V) = v;
        }
        row_h[c] = v;
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(h[i], h[i], ss);
    }
    ss = warp_sum(ss);
    if (lane == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = lane < nt / 32 ? part[lane] : 0.f;
    ss = warp_sum(ss);
    const float rstd = 1.0f / sqrtf(ss / (float)d + eps);

    // (all lanes of a warp take every turn: the block maxima are exchanged between them)
    for (int c0 = threadIdx.x - lane; c0 < nvec; c0 += nt) {
        const int c = c0 + lane;
        const bool in = c < nvec;
        Wide<T> u[V];
        if (in) {
            float h[V], w[V];
            unpack<T>(row_h[c], h);
            unpack<T>(__ldg(reinterpret_cast<const uint4*>(weight) + c), w);
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = (Wide<T>)h[i] * (Wide<T>)w[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = 0;
        }
        if (out_q) {
            const Wide<T> a = group_max(piece_max<T>(u), kLanes<T>);
            float t[V];
            const float scale = block_quotients<T>(u, a, rstd, t);
            if (in) {
                store_values<T>(out_q + at + (int64_t)c * V, t);
                if ((c & (kLanes<T> - 1)) == 0)
                    out_scale[(int64_t)blockIdx.x * ((d + kBlockCols - 1) / kBlockCols) + c / kLanes<T>] = scale;
            }
        }
        if (out_y && in) {
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = (float)(u[i] * (Wide<T>)rstd);
            *reinterpret_cast<uint4*>(out_y + at + (int64_t)c * V) = pack<T>(y);
        }
    }
}

// 1 x 128 blocks: a warp takes 32 pieces of 16 bytes of one row at a time (two blocks of bf16,
// one of float32), kAhead of them with their loads in flight together.
constexpr int kAhead = 4;

template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T* __restrict__ x, int64_t rows, int cols,
                                                            uint8_t* __restrict__ q, float* __restrict__ scale) {
    constexpr int V = kVec<T>;
    const int nvec = cols / V, turns = (nvec + 31) / 32, lane = threadIdx.x & 31;
    const int nblocks = (cols + kBlockCols - 1) / kBlockCols;
    const int64_t units = rows * turns, warps = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t u0 = blockIdx.x * (int64_t)(blockDim.x / 32) + (threadIdx.x >> 5); u0 < units; u0 += kAhead * warps) {
        uint4 v[kAhead];
        int64_t row[kAhead];
        int c[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t unit = u0 + k * warps;
            row[k] = unit / turns;
            c[k] = unit < units ? (int)(unit - row[k] * turns) * 32 + lane : nvec;
            v[k] = c[k] < nvec ? ld_stream_v4(x + row[k] * cols + (int64_t)c[k] * V) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            float f[V], t[V];
            Wide<T> u[V];
            unpack<T>(v[k], f);
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = f[i];
            const Wide<T> a = group_max(piece_max<T>(u), kLanes<T>);
            const float s = block_quotients<T>(u, a, 1.0f, t);
            if (c[k] < nvec) {
                store_values<T>(q + row[k] * cols + (int64_t)c[k] * V, t);
                if ((c[k] & (kLanes<T> - 1)) == 0) scale[row[k] * nblocks + c[k] / kLanes<T>] = s;
            }
        }
    }
}

// 128 x 128 blocks: a CTA of 16 warps holds one in registers
template <typename T>
__global__ void __launch_bounds__(512) quantize_blocks_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                              uint8_t* __restrict__ q, float* __restrict__ scale) {
    constexpr int V = kVec<T>, L = kLanes<T>, N = 128 * L / 512;
    __shared__ float part[16];
    const int64_t nblocks = (cols + kBlockCols - 1) / kBlockCols;
    const int64_t rb = blockIdx.x / nblocks, cb = blockIdx.x - rb * nblocks;
    const int64_t col = cb * kBlockCols + (threadIdx.x % L) * V;
    uint4 v[N];
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t row = rb * 128 + threadIdx.x / L + k * (512 / L);
        v[k] = row < rows && col < cols ? ld_stream_v4(x + row * cols + col) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float f[V];
        unpack<T>(v[k], f);
#pragma unroll
        for (int i = 0; i < V; ++i) a = fmaxf(a, fabsf(f[i]));
    }
    a = warp_max(a);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    a = warp_max(part[threadIdx.x & 15]);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t row = rb * 128 + threadIdx.x / L + k * (512 / L);
        float f[V], t[V];
        Wide<T> u[V];
        unpack<T>(v[k], f);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = f[i];
        const float s = block_quotients<T>(u, (Wide<T>)a, 1.0f, t);
        if (row < rows && col < cols) store_values<T>(q + row * cols + col, t);
        if (k == 0 && threadIdx.x == 0) scale[rb * nblocks + cb] = s;
    }
}

template <typename T>
uno_status norm_launch(const void* x, const void* residual, const void* weight, int64_t M, int64_t d, float eps,
                       void* out_residual, void* out_q, float* out_scale, void* out_y, cudaStream_t stream) {
    const int nvec = (int)d / kVec<T>;
    const int threads = nvec >= kNormThreads ? kNormThreads : (nvec + 31) / 32 * 32;
    const size_t smem = (size_t)nvec * 16;
    if (smem > 48 * 1024) {  // (an attribute of the current device's function: set at each call)
        const uno_status s = check_cuda(
            cudaFuncSetAttribute(norm_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 32768 * (int)sizeof(T)),
            "cudaFuncSetAttribute(rms norm)");
        if (s != UNO_OK) return s;
    }
    norm_kernel<T><<<(unsigned)M, threads, smem, stream>>>(
        static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<const T*>(weight), (int)d, eps,
        static_cast<T*>(out_residual), static_cast<uint8_t*>(out_q), out_scale, static_cast<T*>(out_y));
    return check_cuda(cudaGetLastError(), "launch(rms norm)");
}

template <typename T>
uno_status quantize_launch(const void* x, int64_t rows, int64_t cols, int block_rows, void* q, float* scale,
                           cudaStream_t stream) {
    const int sms = device_sms();
    if (sms == 0) return set_error(UNO_ERR_CUDA, "the current device's properties cannot be read");
    if (block_rows == 1) {
        const int64_t units = rows * ((cols / kVec<T> + 31) / 32);
        const int64_t need = (units + 8 * kAhead - 1) / (8 * kAhead), most = (int64_t)sms * 8;
        quantize_rows_kernel<T><<<(unsigned)(need < most ? need : most), 256, 0, stream>>>(
            static_cast<const T*>(x), rows, (int)cols, static_cast<uint8_t*>(q), scale);
    } else {
        const int64_t blocks = ((rows + 127) / 128) * ((cols + kBlockCols - 1) / kBlockCols);
        if (blocks > 0x7FFFFFFF) return set_error(UNO_ERR_UNSUPPORTED, "more than 2^31 - 1 blocks");
        quantize_blocks_kernel<T><<<(unsigned)blocks, 512, 0, stream>>>(static_cast<const T*>(x), rows, cols,
                                                                       static_cast<uint8_t*>(q), scale);
    }
    return check_cuda(cudaGetLastError(), "launch(fp8 quantize)");
}

}  // namespace
}  // namespace uno

extern "C" uno_status uno_rms_norm_fp8(const void* x, const void* residual, const void* weight, uno_dtype dtype,
                                       int64_t M, int64_t d, float eps, void* out_residual, void* out_q,
                                       float* out_scale, void* out_y, uno_stream_t stream) {
    using namespace uno;
    if (bad_dtype(dtype)) return set_error(UNO_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (M < 0 || d < 1) return set_error(UNO_ERR_INVALID_ARG, "need M >= 0 and d >= 1");
    if (!(eps > 0.f) || !(eps < INFINITY)) return set_error(UNO_ERR_INVALID_ARG, "eps must be positive and finite");
    if (d % 16 || d > 32768) return set_error(UNO_ERR_UNSUPPORTED, "d must be a multiple of 16 and <= 32768");
    if (M > 0x7FFFFFFF) return set_error(UNO_ERR_UNSUPPORTED, "M < 2^31 is supported");
    if (M == 0) return UNO_OK;
    if (!x || !weight) return set_error(UNO_ERR_INVALID_ARG, "x and weight are required");
    if ((out_q == nullptr) != (out_scale == nullptr))
        return set_error(UNO_ERR_INVALID_ARG, "out_q and out_scale are given together");
    if (!out_q && !out_y) return set_error(UNO_ERR_INVALID_ARG, "out_q or out_y is required");
    if (out_residual && !residual) return set_error(UNO_ERR_INVALID_ARG, "out_residual needs residual");
    const void* ptrs[] = {x, residual, weight, out_residual, out_q, out_scale, out_y};
    for (const void* p : ptrs)
        if (off16(p)) return set_error(UNO_ERR_UNSUPPORTED, "tensor pointers must be 16-byte aligned");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == UNO_F32
               ? norm_launch<float>(x, residual, weight, M, d, eps, out_residual, out_q, out_scale, out_y, st)
               : norm_launch<__nv_bfloat16>(x, residual, weight, M, d, eps, out_residual, out_q, out_scale, out_y, st);
}

extern "C" uno_status uno_fp8_quantize(const void* x, uno_dtype dtype, int64_t rows, int64_t cols, int32_t block_rows,
                                       void* out_q, float* out_scale, uno_stream_t stream) {
    using namespace uno;
    if (bad_dtype(dtype)) return set_error(UNO_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (rows < 0 || cols < 1) return set_error(UNO_ERR_INVALID_ARG, "need rows >= 0 and cols >= 1");
    if (block_rows != 1 && block_rows != 128) return set_error(UNO_ERR_INVALID_ARG, "block_rows must be 1 or 128");
    if (cols % 16) return set_error(UNO_ERR_UNSUPPORTED, "cols must be a multiple of 16");
    if (rows > 0x7FFFFFFF || cols > 0x7FFFFFFF)
        return set_error(UNO_ERR_UNSUPPORTED, "rows and cols < 2^31 are supported");
    if (rows == 0) return UNO_OK;
    if (!x || !out_q || !out_scale) return set_error(UNO_ERR_INVALID_ARG, "x, out_q and out_scale are required");
    if (off16(x) || off16(out_q) || off16(out_scale))
        return set_error(UNO_ERR_UNSUPPORTED, "tensor pointers must be 16-byte aligned");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == UNO_F32 ? quantize_launch<float>(x, rows, cols, block_rows, out_q, out_scale, st)
                            : quantize_launch<__nv_bfloat16>(x, rows, cols, block_rows, out_q, out_scale, st);
}
