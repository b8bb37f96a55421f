// fp8_linear.cu — row-gated LoRA linear on an e4m3 base weight (tcgen05).
//
//   Y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in b} xq[m, k] wq[n, k]
//             + scale g[m] sum_j T[m, j] B[n, j],         T = bf16(X A^T)
//
// A K block is 128 bytes of a row: 128 e4m3 columns, or 64 bf16 columns of the adapter's
// (T, B). Each is one tensor-core product into a fresh TMEM accumulator, and the epilogue
// warps add it, times its factor, into float32 registers:
//   e4m3 block b:  acc += xs[m, b] ws[n / 128, b] * D        adapter:  acc += scale g[m] * D
// so scales of any size cost one multiply-add per element and block, and the gate costs
// nothing. T is made by the same kernel first: a product with adapter blocks alone (X, A) and
// factor 1.
//
// A CTA computes a 128 x BN tile (or, in a cluster of S CTAs, its share of the tile's K
// blocks). Warp 0 loads K blocks by TMA into a ring of shared-memory stages; warp 1 issues
// tcgen05.mma into one of NB accumulators; eight epilogue warps (two for each quarter of the
// 128 TMEM lanes, half of the columns each) drain them. The sums then pass through shared
// memory, where the CTAs of a cluster add theirs up in rank order (distributed shared
// memory), and leave as whole rows. Rows past M are never stored; a small M shrinks the
// loaded rows of x, not the product.
//
// Two CTAs fit on an SM (shared memory, TMEM and registers are sized for it): one's prologue,
// drain and stores overlap the other's product.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>

#include "layers.cuh"

namespace uno {
namespace fp8lin {

constexpr int BM = 128;
constexpr int kRowBytes = 128;  // bytes of a K block's row: one 128-byte swizzle row
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxStages = 8;
constexpr int kSmemLimit = 112 * 1024;  // two CTAs per SM
constexpr int kSmemLeast = 78 * 1024;   // and never three: the third's wait for TMEM could hold up a cluster
constexpr int kTmemCols = 256;          // of 512: two CTAs per SM

struct Params {
    int M, N;              // rows and columns of Y
    int nk8, nk16;         // K blocks of e4m3 and of bf16
    int m_tiles;
    int stages;
    uint32_t a_rows;       // rows of x loaded per K block (a multiple of 8, at most 128)
    const float* xs;       // [M, nk8]
    const float* ws;       // [ceil(N / 128), nk8]
    const float* gate;     // [M], or NULL: factor 1 for the bf16 blocks
    float scale;
    void* y;
    int y_f32;
    int wait_t;            // the bf16 blocks' x operand is the previous kernel's output
    uint32_t* status;
};

__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}

// K-major operand with 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 |
           (uint64_t)2u << 61;
}

// instruction descriptors: float32 accumulator, K-major operands; e4m3 x e4m3 or bf16 x bf16
__host__ __device__ constexpr uint32_t shape_bits(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) { return shape_bits(M, N); }
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N) { return shape_bits(M, N) | (1u << 7) | (1u << 10); }

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_load32(uint32_t taddr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t local, uint32_t rank) {
    uint32_t remote;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

// wait for an mbarrier phase (bounded); gives up early once another role of this CTA has
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* gave_up) {
    for (uint32_t i = 0; i < kWaitLimit; i += 256) {
        if (mbar_wait(bar, parity, 256)) return true;
        if (*gave_up) return false;
    }
    return false;
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 2)
linear_kernel(const __grid_constant__ CUtensorMap tX, const __grid_constant__ CUtensorMap tW,
              const __grid_constant__ CUtensorMap tT, const __grid_constant__ CUtensorMap tB, const Params p) {
    constexpr int NB = kTmemCols / BN;  // accumulators
    constexpr int CW = BN / 2;          // columns of an epilogue warp
    constexpr int PITCH = BN + 4;       // floats of a row of sums in shared memory (no bank conflicts)
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], tfull[NB], tempty[NB], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int s_gave_up;

    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
    const int ST = p.stages;
    const uint32_t a_bytes = p.a_rows * kRowBytes;
    constexpr uint32_t b_bytes = BN * kRowBytes;
    const uint32_t ring_b = ring + (uint32_t)ST * a_bytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* gave_up = &s_gave_up;
    const uint32_t S = cluster_size(), rank = cluster_rank();
    const int tile = blockIdx.x / S;
    const int m0 = (tile % p.m_tiles) * BM, n0 = (tile / p.m_tiles) * BN;
    // this CTA's share of the K blocks
    const int nk = p.nk8 + p.nk16;
    const int kb0 = (int)((int64_t)nk * rank / S), kb1 = (int)((int64_t)nk * (rank + 1) / S);

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], kEpiWarps);
        }
        mbar_init(&drain, 1);
        s_gave_up = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base;
    // the next kernel on the stream may start its own prologue (it waits for this grid's end
    // before it reads what this one writes)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    float acc[CW];
    if (warp == 0) {
        if (lane == 0) {
            int s = 0, got = 0;
            uint32_t ph = 1;
            bool waited = !p.wait_t;
            for (int kb = kb0; kb < kb1; ++kb, ++got) {
                if (got >= ST && !wait_phase(&empty[s], ph, gave_up)) {
                    *gave_up = 1;
                    break;
                }
                const bool low = kb >= p.nk8;
                if (low && !waited) {  // T comes from the kernel before this one
                    asm volatile("griddepcontrol.wait;\n\tfence.proxy.async.global;" ::: "memory");
                    waited = true;
                }
                mbar_arrive_expect_tx(&full[s], a_bytes + b_bytes);
                const uint32_t a = ring + (uint32_t)s * a_bytes, b = ring_b + (uint32_t)s * b_bytes;
                if (low) {
                    load_2d(a, &tT, (kb - p.nk8) * 64, m0, &full[s]);
                    load_2d(b, &tB, (kb - p.nk8) * 64, n0, &full[s]);
                } else {
                    load_2d(a, &tX, kb * 128, m0, &full[s]);
                    load_2d(b, &tW, kb * 128, n0, &full[s]);
                }
                if (++s == ST) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (*gave_up)  // loads that no product will read: let them land
                for (int j = got > ST ? got - ST : 0; j < got; ++j) mbar_wait(&full[j % ST], (j / ST) & 1, 1u << 16);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint64_t da0 = operand_desc(ring), db0 = operand_desc(ring_b);
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 1;
            for (int kb = kb0; kb < kb1; ++kb) {
                if ((kb - kb0 >= NB && !wait_phase(&tempty[b], bph, gave_up)) || !wait_phase(&full[s], ph, gave_up)) {
                    *gave_up = 1;
                    break;
                }
                fence_after();
                const uint64_t da = da0 + (uint64_t)(((uint32_t)s * a_bytes) >> 4);
                const uint64_t db = db0 + (uint64_t)(((uint32_t)s * b_bytes) >> 4);
                const uint32_t d = tmem + (uint32_t)(b * BN);
                if (kb < p.nk8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 32 bytes of K per instruction
                        mma_e4m3(d, da + 2 * k, db + 2 * k, idesc_e4m3(BM, BN), k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_bf16(d, da + 2 * k, db + 2 * k, idesc_bf16(BM, BN), k > 0);
                }
                commit(&empty[s]);
                commit(&tfull[b]);
                if (++s == ST) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++b == NB) {
                    b = 0;
                    bph ^= 1u;
                }
            }
            if (*gave_up) {  // products in flight end before their memory is given back
                commit(&drain);
                mbar_wait(&drain, 0, 1u << 16);
            }
        }
    } else {
        // ---- epilogue: acc += factor * accumulator, one row a thread, CW columns ----
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const int row = m0 + quarter * 32 + lane;
        const bool any = m0 + quarter * 32 < p.M;  // (a warp of rows past M only keeps the barriers going)
        const float* xs = p.xs + (int64_t)(row < p.M ? row : 0) * p.nk8;
        const float* ws = p.ws + (int64_t)(n0 / kBlockCols) * p.nk8;
        const float low = p.gate ? (row < p.M ? p.scale * p.gate[row] : 0.f) : 1.f;
#pragma unroll
        for (int j = 0; j < CW; ++j) acc[j] = 0.f;
        int b = 0;
        uint32_t bph = 0;
        float f4[4];
        for (int kb = kb0; kb < kb1; ++kb) {
            const int at = (kb - kb0) & 3;
            if (at == 0 && any) {  // the factors of the next four K blocks
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f4[j] = kb + j < p.nk8 ? __ldg(xs + kb + j) * __ldg(ws + kb + j) : low;
            }
            if (!__all_sync(kFullMask, wait_phase(&tfull[b], bph, gave_up))) {
                *gave_up = 1;
                break;
            }
            fence_after();
            if (any) {
                const float f = at == 0 ? f4[0] : at == 1 ? f4[1] : at == 2 ? f4[2] : f4[3];
                const bool off = kb >= p.nk8 && f == 0.f;  // no adapter on this row, whatever its product holds
                const uint32_t taddr = tmem + (uint32_t)(b * BN + half * CW) + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
                for (int c = 0; c < CW; c += 32) {
                    float r[32];
                    __syncwarp();
                    tmem_load32(taddr + (uint32_t)c, r);
                    if (!off) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(f, r[j], acc[c + j]);
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[b]);
            if (++b == NB) {
                b = 0;
                bph ^= 1u;
            }
        }
    }

    // ---- the tile's sums, through shared memory (the ring: every product has read its stage) ----
    fence_before();
    __syncthreads();
    fence_after();
    const int rows = p.M - m0 < BM ? p.M - m0 : BM;
    if (warp >= 2) {
        const int quarter = warp & 3, half = (warp - 2) >> 2, r = quarter * 32 + lane;
        if (r < rows) {
            const uint32_t at = ring + (uint32_t)(r * PITCH + half * CW) * 4u;
#pragma unroll
            for (int j = 0; j < CW; j += 4)
                asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at + j * 4u), "f"(acc[j]), "f"(acc[j + 1]),
                             "f"(acc[j + 2]), "f"(acc[j + 3])
                             : "memory");
        }
    }
    __syncwarp();
    if (S > 1) cluster_sync();
    else __syncthreads();
    if (!*gave_up) {
        // rank r of the cluster writes its share of the rows
        const int r0 = (int)(rows * rank / S), r1 = (int)(rows * (rank + 1) / S);
        const bool vec = p.N % 8 == 0;  // rows start on 16 bytes
        for (int i = threadIdx.x; i < (r1 - r0) * (BN / 8); i += kThreads) {
            const int r = r0 + i / (BN / 8), c = (i % (BN / 8)) * 8;
            const int col = n0 + c;
            if (col >= p.N) continue;
            float v[8] = {};
            const uint32_t at = ring + (uint32_t)(r * PITCH + c) * 4u;
            for (uint32_t k = 0; k < S; ++k) {
                const float4 lo = ld_cluster(at, k), hi = ld_cluster(at + 16u, k);
                v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w;
                v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
            }
            const int64_t o = (int64_t)(m0 + r) * p.N + col;
            if (p.y_f32) {
                float* y = static_cast<float*>(p.y) + o;
                if (vec) {
                    reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
                    reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col + j < p.N) y[j] = v[j];
                }
            } else {
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + o;
                if (vec) {
                    *reinterpret_cast<uint4*>(y) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col + j < p.N) y[j] = __float2bfloat16_rn(v[j]);
                }
            }
        }
    }
    __syncwarp();
    if (S > 1) cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
    if (threadIdx.x == 0 && *gave_up) record_device_status(p.status, (uint32_t)UNO_ERR_TIMEOUT);
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
    auto f = fn.load(std::memory_order_acquire);
    if (!f) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
            fn.store(f, std::memory_order_release);
        }
    }
    return f;
}

// row-major [rows, cols] matrix, boxes of 128 bytes of columns x box_rows rows, 128-byte swizzle
uno_status operand_map(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, bool bf16, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return set_error(UNO_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t gstride[1] = {(cuuint64_t)cols * (bf16 ? 2 : 1)};
    const cuuint32_t box[2] = {bf16 ? 64u : 128u, box_rows};
    const cuuint32_t step[2] = {1, 1};
    const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                          const_cast<void*>(ptr), gdim, gstride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(UNO_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return UNO_OK;
}

struct Shape {
    int BN, S, stages;
    uint32_t a_rows;
    size_t smem;
};

// Tile width, CTAs per tile and ring depth of a product of M x N with nk K blocks.
Shape choose(int64_t M, int64_t N, int nk, int sms) {
    Shape c{};
    c.a_rows = M >= BM ? BM : (uint32_t)((M + 7) / 8 * 8);
    const int64_t m_tiles = (M + BM - 1) / BM;
    c.BN = m_tiles * ((N + 127) / 128) * 8 < sms ? 64 : 128;
    const int64_t tiles = m_tiles * ((N + c.BN - 1) / c.BN);
    c.S = 1;
    while (c.S < 8 && tiles * c.S * 2 <= 2 * sms && nk >= c.S * 4) c.S *= 2;
    const uint32_t stage = (c.a_rows + c.BN) * kRowBytes;
    const uint32_t sums = BM * (uint32_t)(c.BN + 4) * 4u;
    c.stages = (int)((kSmemLimit - 1024) / stage);
    if (c.stages > kMaxStages) c.stages = kMaxStages;
    // the product reads 128 rows of x from every stage, loaded or not
    size_t need = (size_t)c.stages * stage;
    if (need < (size_t)(c.stages - 1) * c.a_rows * kRowBytes + BM * kRowBytes)
        need = (size_t)(c.stages - 1) * c.a_rows * kRowBytes + BM * kRowBytes;
    if (need < sums) need = sums;
    if (need < kSmemLeast) need = kSmemLeast;
    c.smem = need + 1024;
    return c;
}

template <int BN>
uno_status launch(const Shape& c, const CUtensorMap (&maps)[4], const Params& p, int64_t tiles, bool overlap,
                  cudaStream_t stream) {
    uno_status s = check_cuda(cudaFuncSetAttribute(linear_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kSmemLimit + 1024),
                              "cudaFuncSetAttribute(fp8 linear)");
    if (s != UNO_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3((unsigned)(tiles * c.S));
    cfg.dynamicSmemBytes = c.smem;
    cfg.stream = stream;
    cfg.attrs = attrs;
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = (unsigned)c.S;
    attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = overlap ? 2 : 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, linear_kernel<BN>, maps[0], maps[1], maps[2], maps[3], p),
                      "launch(fp8 linear)");
}

// one product: e4m3 blocks over d_in columns (or none), bf16 blocks over r columns (or none)
uno_status product(const void* xq, const void* wq, int64_t d_in, const void* t, const void* b, int64_t r, Params p,
                   bool overlap, cudaStream_t stream) {
    const int sms = device_sms();
    p.status = device_status_ptr();
    if (sms == 0 || !p.status) return set_error(UNO_ERR_CUDA, "the current device's properties cannot be read");
    p.nk8 = (int)((d_in + 127) / 128);
    p.nk16 = (int)((r + 63) / 64);
    const Shape c = choose(p.M, p.N, p.nk8 + p.nk16, sms);
    p.m_tiles = (p.M + BM - 1) / BM;
    p.stages = c.stages;
    p.a_rows = c.a_rows;
    const int64_t tiles = (int64_t)p.m_tiles * ((p.N + c.BN - 1) / c.BN);
    if (tiles * c.S > 0x7FFFFFFF) return set_error(UNO_ERR_UNSUPPORTED, "too many output tiles");
    CUtensorMap maps[4];
    uno_status s = UNO_OK;
    if (d_in) {
        s = operand_map(&maps[0], xq, p.M, d_in, false, c.a_rows);
        if (s == UNO_OK) s = operand_map(&maps[1], wq, p.N, d_in, false, (uint32_t)c.BN);
    }
    if (s == UNO_OK && r) {
        s = operand_map(&maps[2], t, p.M, r, true, c.a_rows);
        if (s == UNO_OK) s = operand_map(&maps[3], b, p.N, r, true, (uint32_t)c.BN);
    }
    if (s != UNO_OK) return s;
    if (!d_in) maps[0] = maps[2], maps[1] = maps[3];  // (not read)
    if (!r) maps[2] = maps[0], maps[3] = maps[1];
    return c.BN == 64 ? launch<64>(c, maps, p, tiles, overlap, stream)
                      : launch<128>(c, maps, p, tiles, overlap, stream);
}

}  // namespace fp8lin
}  // namespace uno

extern "C" size_t uno_fp8_gated_lora_linear_workspace_size(int64_t M, int64_t d_in, int64_t d_out, int64_t rank) {
    if (M < 1 || d_in < 1 || d_out < 1 || rank < 1) return 0;
    return uno::align_up((size_t)M * (size_t)rank * 2, 256);  // T
}

extern "C" uno_status uno_fp8_gated_lora_linear(const void* x_q, const float* x_scale, const void* w_q,
                                                const float* w_scale, const void* x, const void* lora_a,
                                                const void* lora_b, const float* row_gate, float scale, int64_t M,
                                                int64_t d_in, int64_t d_out, int64_t rank, void* y, uno_dtype y_dtype,
                                                void* workspace, size_t workspace_bytes, uno_stream_t stream) {
    using namespace uno;
    if (bad_dtype(y_dtype)) return set_error(UNO_ERR_INVALID_ARG, "unknown dtype %d", (int)y_dtype);
    if (M < 0 || d_in < 1 || d_out < 1 || rank < 0)
        return set_error(UNO_ERR_INVALID_ARG, "need M >= 0, d_in >= 1, d_out >= 1, rank >= 0");
    if (d_in % 16 || d_in > 65536 || d_out > (1 << 20) || M > (1 << 20))
        return set_error(UNO_ERR_UNSUPPORTED, "d_in a multiple of 16 up to 65536, d_out and M up to 2^20 are supported");
    if (rank % 8 || rank > 256) return set_error(UNO_ERR_UNSUPPORTED, "rank must be 0 or a multiple of 8 and <= 256");
    if (rank && y_dtype == UNO_F32) return set_error(UNO_ERR_UNSUPPORTED, "float32 output is supported with rank 0");
    if (M == 0) return UNO_OK;
    if (!x_q || !x_scale || !w_q || !w_scale || !y) return set_error(UNO_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (rank && (!x || !lora_a || !lora_b)) return set_error(UNO_ERR_INVALID_ARG, "rank > 0 needs x, lora_a and lora_b");
    if (rank && !(std::isfinite(scale))) return set_error(UNO_ERR_INVALID_ARG, "scale must be finite");
    const void* ptrs[] = {x_q, x_scale, w_q, w_scale, y};
    for (const void* p : ptrs)
        if (off16(p)) return set_error(UNO_ERR_UNSUPPORTED, "tensor pointers must be 16-byte aligned");
    if (rank && (off16(x) || off16(lora_a) || off16(lora_b) || off16(row_gate)))
        return set_error(UNO_ERR_UNSUPPORTED, "tensor pointers must be 16-byte aligned");
    const bool adapter = rank > 0 && row_gate != nullptr;  // without a gate no row has one
    const size_t need = uno_fp8_gated_lora_linear_workspace_size(M, d_in, d_out, rank);
    if (need) {
        if (!workspace) return set_error(UNO_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
        if (reinterpret_cast<uintptr_t>(workspace) & 255u)
            return set_error(UNO_ERR_WORKSPACE, "workspace not 256-byte aligned");
        if (workspace_bytes < need)
            return set_error(UNO_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    fp8lin::Params p{};
    p.M = (int)M;
    if (adapter) {  // T = bf16(X A^T)
        fp8lin::Params t = p;
        t.N = (int)rank;
        t.y = workspace;
        const uno_status s = fp8lin::product(nullptr, nullptr, 0, x, lora_a, d_in, t, false, st);
        if (s != UNO_OK) return s;
    }
    p.N = (int)d_out;
    p.xs = x_scale;
    p.ws = w_scale;
    p.gate = adapter ? row_gate : nullptr;
    p.scale = scale;
    p.y = y;
    p.y_f32 = y_dtype == UNO_F32;
    p.wait_t = adapter;
    return fp8lin::product(x_q, w_q, d_in, workspace, lora_b, adapter ? rank : 0, p, adapter, st);
}
