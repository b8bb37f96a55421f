// norm_fp8.cu — RMS norm with the residual's addition and e4m3 output, and the e4m3
// quantiser of weights and activations.
//
//   h = x + residual,  u = h * weight,  rstd = 1 / sqrt(mean h^2 + eps),  y = u rstd
//   per block, a = max |u|:  scale = max(a rstd / 448, 2^-126),  value = e4m3(448 u / a)
// The row's factor rstd cancels in the values, so they need no statistics: only the scales
// do. The quotient 448 u / a is what is rounded, once, to nearest even:
// Found in float32 as u c + u r, with c near 448 / a and r its remainder, it is off by its last
// rounding, 2^-24, and no more:
//   bf16 inputs: u is exact in float32 (a product of two 8-bit significands), but for products below
//     its normal numbers or beyond it, which the norm takes as float32 has them. 448 u and
//     border * a are whole numbers of at most 21 bits on a common scale, so a quotient that is
//     not on a border of e4m3 is at least 2^-21 away from it, and one that is on it comes out
//     exactly: the values are those of exact arithmetic.
//   float32 inputs of the quantiser: 2^-32 away at least. A quotient that came out on a border
//     is moved by one unit to the side on which its remainder says that it lies.
//   float32 inputs of the norm: u takes 48 bits; float64, rounded to float32 to odd so that the
//     second rounding, to e4m3, sees on which side of a border the quotient lies.
//
// Bound: HBM. The norm reads x and the residual and writes h, the values and, if asked, y,
// each once; a row is held in shared memory between its sum of squares and its values (16
// bytes a thread at a time, read back by the thread that wrote them). One CTA per row.
// Measured: the norm of 16384 x 2560 with a residual 51 us, 5.8 TB/s, in bf16 and 105 us, 5.2 TB/s,
// in float32; of 16 x 4096 2.4 and 3.8 us (one row's latency); the quantiser on 1024 x 12288 float32
// 14.4 us, 4.4 TB/s, and on 9728 x 2560 by 128 x 128 blocks 14.6 us, 5.1 TB/s, in bf16 and 24.4 us,
// 5.1 TB/s, in float32 (sizes near that of L2, a launch's ramp in each).
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

constexpr int V = 8;                     // values a lane takes at a time
constexpr int kLanes = kBlockCols / V;   // lanes that hold one 128-column block

// V values of a row in their storage type: 16 bytes of bf16, 32 of float32
template <typename T>
struct Piece {
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Piece<T> zero_piece() {
    Piece<T> v;
#pragma unroll
    for (auto& w : v.w) w = make_uint4(0, 0, 0, 0);
    return v;
}
template <typename T>
__device__ __forceinline__ Piece<T> load_piece(const T* p) {
    Piece<T> v;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v.w[i] = reinterpret_cast<const uint4*>(p)[i];
    return v;
}
template <typename T>
__device__ __forceinline__ Piece<T> stream_piece(const T* p) {
    Piece<T> v;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v.w[i] = ld_stream_v4(p + i * 4);
    return v;
}
template <typename T>
__device__ __forceinline__ void store_piece(T* p, const Piece<T>& v) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = v.w[i];
}

template <typename T>
__device__ __forceinline__ void unpack(const Piece<T>& v, float (&f)[V]) {
    if constexpr (std::is_same_v<T, float>) {
        const uint32_t w[8] = {v.w[0].x, v.w[0].y, v.w[0].z, v.w[0].w, v.w[1].x, v.w[1].y, v.w[1].z, v.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else {
        const uint32_t w[4] = {v.w[0].x, v.w[0].y, v.w[0].z, v.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <typename T>
__device__ __forceinline__ Piece<T> pack(const float (&f)[V]) {
    Piece<T> v;
    if constexpr (std::is_same_v<T, float>) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v.w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                                __float_as_uint(f[4 * i + 3]));
    } else {
        v.w[0] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
    return v;
}

// the largest over the kLanes lanes that hold a block
template <typename U>
__device__ __forceinline__ U group_max(U v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
        v = fmax(v, __shfl_xor_sync(kFullMask, v, o));
    }
    return v;
}

// of the stored bf16 values two at a time; the low half's largest and the high half's join last
__device__ __forceinline__ float group_max_bf16(const Piece<__nv_bfloat16>& v) {
    auto half2 = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
    __nv_bfloat162 m = __hmax2(__hmax2(__habs2(half2(v.w[0].x)), __habs2(half2(v.w[0].y))),
                               __hmax2(__habs2(half2(v.w[0].z)), __habs2(half2(v.w[0].w))));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        m = __hmax2(m, half2(__shfl_xor_sync(kFullMask, *reinterpret_cast<uint32_t*>(&m), o)));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.f);  // (0 where all are NaN)
}

template <typename U>
__device__ __forceinline__ U piece_max(const U (&u)[V]) {
    U a = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) a = fmax(a, fabs(u[i]));  // (a NaN is passed over)
    return a;
}

__device__ __forceinline__ float reciprocal(float a) {  // within an ulp or two
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

// float64 to float32, to odd: a value between two float32 numbers goes to the one whose last
// bit is set, so rounding the result again to a much shorter type rounds the value itself
__device__ __forceinline__ float to_odd(double t) {
    const uint32_t inexact = (__double2loint(t) & 0x1FFFFFFF) != 0 ? 1u : 0u;
    return __uint_as_float(__float_as_uint(__double2float_rz(t)) | inexact);
}

// 448 / a in float64 (a number and its remainder) for a block whose largest size is a, in a row
// whose factor is `factor`; the smallest scale and every range of a.
struct Inverse64 {
    double c, r;
};
__device__ __noinline__ Inverse64 inverse64(double a, float factor) {
    double top = a;
    if ((float)(a * (double)factor / 448.0) < kMinScale) {
        const double least = 448.0 * (double)kMinScale / (double)factor;
        top = top > least ? top : least;
    }
    const double c = 448.0 / top;
    return {c, fma(-c, top, 448.0) / top};
}
__device__ __forceinline__ float scale64(double a, float factor) {
    const float scale = (float)(a * (double)factor * (1.0 / 448.0));
    return scale < kMinScale ? kMinScale : scale;
}

// u c + u r of two values
__device__ __forceinline__ void scaled2(float u0, float u1, float c, float r, float& t0, float& t1) {
    uint64_t u, cc, rr, t;
    asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(u0), "f"(u1));
    asm("mov.b64 %0, {%1, %1};" : "=l"(cc) : "f"(c));
    asm("mov.b64 %0, {%1, %1};" : "=l"(rr) : "f"(r));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(u), "l"(rr));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t) : "l"(u), "l"(cc));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(t0), "=f"(t1) : "l"(t));
}

// The same for u that float32 holds exactly. EXACT: 448 u / a is known not to lie within
// 2^-24 of a border of e4m3 without being on it (see above). ORDINARY: a is known to be far from
// overflow and underflow.
template <bool EXACT, bool ORDINARY = false>
__device__ __forceinline__ float quotients(const float (&u)[V], float a, float factor, float (&t)[V]) {
    // a factor / 448, the 1 / 448 as a float32 and its remainder (one rounding where factor is 1)
    constexpr float hi = (float)(1.0 / 448.0), lo = (float)(1.0 / 448.0 - (double)hi);
    const float y = a * factor, scale = fmaf(y, hi, y * lo);
    // far from overflow and underflow of 448 / a and its remainder
    if (ORDINARY || (a >= 0x1p-90f && a <= 0x1p90f && scale >= kMinScale)) {
        const float inv = reciprocal(a), c = kE4m3Max * inv;
        const float r = fmaf(-c, a, kE4m3Max) * inv;  // 448 / a - c, to 20 bits and more
#pragma unroll
        for (int i = 0; i < V; i += 2) scaled2(u[i], u[i + 1], c, r, t[i], t[i + 1]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!EXACT && (__float_as_uint(t[i]) & 0x7FFFFu) == 0u) {
                // on a border, or rounded to it: to the side on which the quotient lies
                const float e = fmaf(u[i], c, -t[i]) + u[i] * r;
                if (fabsf(e) > 0x1p-40f * fabsf(t[i]))
                    t[i] = __uint_as_float(__float_as_uint(t[i]) + ((e > 0.f) == (t[i] > 0.f) ? 1u : ~0u));
            }
        }
        return scale;
    }
    if (a == 0.f) {  // nothing but zeros and NaN
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = u[i];
        return factor == factor ? kMinScale : factor;
    }
    const Inverse64 w = inverse64(a, factor);
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = to_odd(fma((double)u[i], w.c, (double)u[i] * w.r));
    return scale64(a, factor);
}

__device__ __forceinline__ uint2 values(const float (&t)[V]) {
    return make_uint2(e4m3x4(t[0], t[1], t[2], t[3]), e4m3x4(t[4], t[5], t[6], t[7]));
}

// The values and the scale of this lane's piece of a block (all lanes of a block together)
template <typename T>
__device__ __forceinline__ uint2 block_values(const Piece<T>& v, float& scale) {
    float f[V], t[V], a;
    unpack<T>(v, f);
    if constexpr (std::is_same_v<T, float>) a = group_max(piece_max(f));
    else a = group_max_bf16(v);
    scale = quotients<!std::is_same_v<T, float>>(f, a, 1.0f, t);
    return values(t);
}

constexpr int kNormThreads = 512;
template <typename T>
constexpr int kNormAhead = std::is_same_v<T, float> ? 2 : 4;  // pieces with their loads in flight together

// (x and residual may be out_residual: no restrict, no read-only loads. A thread reads its
// piece before it writes it.)
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const T* x, const T* residual, const T* __restrict__ weight,
                                                            int d, float eps, T* out_residual,
                                                            uint8_t* __restrict__ out_q, float* __restrict__ out_scale,
                                                            T* __restrict__ out_y) {
    extern __shared__ uint4 row_raw[];
    Piece<T>* row_h = reinterpret_cast<Piece<T>*>(row_raw);
    __shared__ float part[kNormThreads / 32];
    const int nvec = d / V, nt = blockDim.x, lane = threadIdx.x & 31;
    const int64_t at = (int64_t)blockIdx.x * d;
    float ss = 0.f;
    for (int c0 = threadIdx.x; c0 < nvec; c0 += kNormAhead<T> * nt) {
        Piece<T> v[kNormAhead<T>], r[kNormAhead<T>];
#pragma unroll
        for (int k = 0; k < kNormAhead<T>; ++k) {
            const int c = c0 + k * nt;
            if (c < nvec) v[k] = load_piece(x + at + c * V);
            if (c < nvec && residual) r[k] = load_piece(residual + at + c * V);
        }
#pragma unroll
        for (int k = 0; k < kNormAhead<T>; ++k) {
            const int c = c0 + k * nt;
            if (c >= nvec) break;
            float h[V];
            unpack<T>(v[k], h);
            if (residual) {
                float f[V];
                unpack<T>(r[k], f);
#pragma unroll
                for (int i = 0; i < V; ++i) h[i] += f[i];
                v[k] = pack<T>(h);
                unpack<T>(v[k], h);  // the rounded sum is what is normed
                if (out_residual) store_piece(out_residual + at + c * V, v[k]);
            }
            row_h[c] = v[k];
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(h[i], h[i], ss);
        }
    }
    ss = warp_sum(ss);
    if (lane == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < nt / 32; ++w) ss += part[w];
    // (the approximation and a Newton step: within 2^-23)
    const float ms = ss / (float)d + eps;
    float rstd = rsqrtf(ms);
    rstd = fmaf(rstd * 0.5f, fmaf(-ms * rstd, rstd, 1.0f), rstd);

    // (all lanes of a warp take every turn: the block maxima are exchanged between them)
    for (int c0 = threadIdx.x - lane; c0 < nvec; c0 += nt) {
        const int c = c0 + lane;
        const bool in = c < nvec;
        float h[V], w[V], t[V], scale = 0.f;
        unpack<T>(in ? row_h[c] : zero_piece<T>(), h);
        unpack<T>(in ? load_piece(weight + c * V) : zero_piece<T>(), w);
        if constexpr (std::is_same_v<T, float>) {
            double u[V];
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = (double)h[i] * (double)w[i];
            if (out_q) {
                const double a = group_max(piece_max(u));
                const Inverse64 w64 = inverse64(a, rstd);
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] = to_odd(fma(u[i], w64.c, u[i] * w64.r));
                scale = scale64(a, rstd);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] = (float)(u[i] * (double)rstd);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] *= w[i];
            if (out_q) scale = quotients<true>(h, group_max(piece_max(h)), rstd, t);
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] *= rstd;
        }
        if (!in) continue;
        if (out_q) {
            *reinterpret_cast<uint2*>(out_q + at + c * V) = values(t);
            if (c % kLanes == 0) out_scale[(int64_t)blockIdx.x * ((nvec + kLanes - 1) / kLanes) + c / kLanes] = scale;
        }
        if (out_y) store_piece(out_y + at + c * V, pack<T>(h));
    }
}

// 1 x 128 blocks where rows end between blocks (cols a multiple of 128): the matrix is one run
// of blocks, whatever its rows. A warp takes two blocks (32 pieces) at a time, kAhead times
// that with the loads in flight together.
// Each thread does kAhead pieces, once: CTAs that loop leave a part of their last turn empty.
template <typename T>
constexpr int kAhead = std::is_same_v<T, float> ? 2 : 4;  // (64 bytes)

template <typename T>
__global__ void __launch_bounds__(256) quantize_run_kernel(const T* __restrict__ x, int64_t pieces,
                                                           uint8_t* __restrict__ q, float* __restrict__ scale) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i - (int64_t)(threadIdx.x & 31) < pieces;
         i += kAhead<T> * step) {
        Piece<T> v[kAhead<T>];
#pragma unroll
        for (int k = 0; k < kAhead<T>; ++k)
            v[k] = i + k * step < pieces ? stream_piece(x + (i + k * step) * V) : zero_piece<T>();
#pragma unroll
        for (int k = 0; k < kAhead<T>; ++k) {
            const int64_t at = i + k * step;
            if (at - (threadIdx.x & 31) >= pieces) break;  // (the whole warp)
            float s;
            const uint2 e = block_values<T>(v[k], s);
            if (at < pieces) {
                *reinterpret_cast<uint2*>(q + at * V) = e;
                if (threadIdx.x % kLanes == 0) scale[at / kLanes] = s;
            }
        }
    }
}

// 1 x 128 blocks with a short last block in each row: a warp takes 32 pieces of one row at a
// time. The unit after the next `warps` is found by adding their quotient and remainder by the
// row's units: no division in the loop.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T* __restrict__ x, int64_t rows, int cols,
                                                            uint8_t* __restrict__ q, float* __restrict__ scale) {
    const int nvec = cols / V, turns = (nvec + 31) / 32, lane = threadIdx.x & 31;
    const int nblocks = (nvec + kLanes - 1) / kLanes;
    const uint32_t warps = gridDim.x * (blockDim.x / 32), first = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    const int64_t more_rows = warps / turns;
    const int more_turns = (int)(warps % turns);
    int64_t row = first / turns;
    int turn = (int)(first % turns);
    while (row < rows) {
        Piece<T> v[kAhead<T>];
        int64_t at[kAhead<T>];
        int c[kAhead<T>];
#pragma unroll
        for (int k = 0; k < kAhead<T>; ++k) {
            at[k] = row;
            c[k] = row < rows ? turn * 32 + lane : nvec;
            v[k] = c[k] < nvec ? stream_piece(x + row * cols + c[k] * V) : zero_piece<T>();
            row += more_rows;
            turn += more_turns;
            if (turn >= turns) {
                turn -= turns;
                ++row;
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead<T>; ++k) {
            if (at[k] >= rows) break;
            float s;
            const uint2 e = block_values<T>(v[k], s);
            if (c[k] < nvec) {
                *reinterpret_cast<uint2*>(q + at[k] * cols + c[k] * V) = e;
                if (c[k] % kLanes == 0) scale[at[k] * nblocks + c[k] / kLanes] = s;
            }
        }
    }
}

// 128 x 128 blocks: a CTA holds one in registers, four or eight pieces a thread. Its loads, its
// maximum and its stores come one after the other, so other CTAs have to fill the gaps: three of
// 256 threads an SM take 14.6 us for 9728 x 2560 bf16, two of 512 16.8 (float32, whose pieces take
// twice the registers: two of 512 23.4, of 256 26.9).
template <typename T>
constexpr int kBlockThreads = std::is_same_v<T, float> ? 512 : 256;
template <typename T>
constexpr int kBlockCtas = std::is_same_v<T, float> ? 2 : 3;  // per SM, as registers allow
template <typename T>
__global__ void __launch_bounds__(kBlockThreads<T>, kBlockCtas<T>)
quantize_blocks_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, uint8_t* __restrict__ q,
                       float* __restrict__ scale) {
    constexpr int NT = kBlockThreads<T>, N = 128 * kLanes / NT;
    __shared__ float part[NT / 32];
    const int64_t nblocks = (cols + kBlockCols - 1) / kBlockCols;
    const int64_t rb = blockIdx.x / nblocks, cb = blockIdx.x - rb * nblocks;
    const int64_t col = cb * kBlockCols + (threadIdx.x % kLanes) * V, row0 = rb * 128 + threadIdx.x / kLanes;
    Piece<T> v[N];
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t row = row0 + k * (NT / kLanes);
        v[k] = row < rows && col < cols ? stream_piece(x + row * cols + col) : zero_piece<T>();
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float f[V];
        unpack<T>(v[k], f);
        a = fmaxf(a, piece_max(f));
    }
    a = warp_max(a);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    a = warp_max(part[threadIdx.x & (NT / 32 - 1)]);
    uint8_t* out = q + row0 * cols + col;
    const bool in = col < cols;
    const int left = in ? (int)(rows - row0 < 128 ? rows - row0 : 128) : 0;  // of this thread's rows
    auto each = [&](auto ordinary) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float f[V], t[V];
            unpack<T>(v[k], f);
            s = quotients<!std::is_same_v<T, float>, decltype(ordinary)::value>(f, a, 1.0f, t);
            if (k * (NT / kLanes) < left) *reinterpret_cast<uint2*>(out + k * (NT / kLanes) * cols) = values(t);
        }
        if (threadIdx.x == 0) scale[rb * nblocks + cb] = s;
    };
    if (a >= 0x1p-90f && a <= 0x1p90f) each(std::true_type{});
    else each(std::false_type{});
}

template <typename T>
uno_status norm_launch(const void* x, const void* residual, const void* weight, int64_t M, int64_t d, float eps,
                       void* out_residual, void* out_q, float* out_scale, void* out_y, cudaStream_t stream) {
    const int nvec = (int)d / V;
    // a piece a thread where rows are few and the call's length is a row's latency; else CTAs of
    // four warps, whose barriers hold up less (M 4096, d 4096, bf16: 16.5 us against 21.5 with
    // eight warps and 32.7 with sixteen)
    int threads = (nvec + 31) / 32 * 32;
    const int most = M >= 4 * (int64_t)device_sms() ? 128 : kNormThreads;
    if (threads > most) threads = most;
    const size_t smem = (size_t)nvec * sizeof(Piece<T>);
    // a launch has 48 KB without asking, its static part (`part`, and alignment) included. (An attribute
    // of the current device's function: set at each call.)
    if (smem > 47 * 1024) {
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
    if (block_rows == 1) {
        const int64_t units = rows * ((cols / V + 31) / 32);  // (a warp's share of a turn)
        const int64_t need = (units + 8 * kAhead<T> - 1) / (8 * kAhead<T>);
        const unsigned grid = (unsigned)(need < (1 << 26) ? need : 1 << 26);
        const T* src = static_cast<const T*>(x);
        uint8_t* dst = static_cast<uint8_t*>(q);
        if (cols % kBlockCols == 0)
            quantize_run_kernel<T><<<grid, 256, 0, stream>>>(src, rows * (cols / V), dst, scale);
        else
            quantize_rows_kernel<T><<<grid, 256, 0, stream>>>(src, rows, (int)cols, dst, scale);
    } else {
        const int64_t blocks = ((rows + 127) / 128) * ((cols + kBlockCols - 1) / kBlockCols);
        if (blocks > 0x7FFFFFFF) return set_error(UNO_ERR_UNSUPPORTED, "more than 2^31 - 1 blocks");
        quantize_blocks_kernel<T><<<(unsigned)blocks, kBlockThreads<T>, 0, stream>>>(
            static_cast<const T*>(x), rows, cols, static_cast<uint8_t*>(q), scale);
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
