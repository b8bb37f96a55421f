// fp8_linear.cu — row-gated LoRA linear on an e4m3 base weight (tcgen05).
//
//   Y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in b} xq[m, k] wq[n, k]
//             + scale g[m] sum_j T[m, j] B[n, j],         T = bf16(X A^T)
//
// A K block is 128 bytes of a row: 128 e4m3 columns, or 64 bf16 columns of the adapter's
// (T, B). Each is one tensor-core product into a fresh TMEM accumulator, and the epilogue
// warps add it, times its factor, into float32 registers:
//   e4m3 block b:  acc += xs[m, b] ws[n / 128, b] * D        adapter:  acc += scale g[m] * D
// so the scales cost one multiply-add per element and block, whatever they are (xs ws is a float32
// product, rounded once; below 2^-126 it keeps fewer bits), and the gate costs nothing.
// T is rounded to bf16 because its product with B takes operands of one type (uno_gated_lora_linear
// rounds its own too). Against 64 bits that is a small part of what Y's rounding is: all differences
// of Y come to 1.8e-3 of its size with it and 1.7e-3 without (M 16 and M 1024). T in two bf16 parts
// would double the adapter's K blocks.
// T is made by the same kernel first: a product with adapter blocks alone (X, A) and
// factor 1; the projection is launched to start on the SMs that this leaves free, and waits for
// its end before it reads T (M 16, 4096 -> 4096, rank 128: 13.5 us, 19.1 one after the other).
//
// Bound: tensor cores and draining for large M (M 8192, 2560 -> 9728: 214 us, 1907 TFLOP/s), HBM
// for few rows of a wide head (M 64, 4096 -> 151936: 113 us, 5.7 TB/s), and between them the draining
// chain of a tile's K blocks (M 16, 4096 -> 4096 without an adapter: 9.5 us for 17 MB from HBM,
// 8.3 from L2). These are at 1965 MHz, as a burst finds the SMs; the power limit lowers the clock
// of a second of the same to 1575 MHz, and times follow it: 245 and 133 us.
//
// Roles of a CTA's warps: 0 loads K blocks by TMA into a ring of shared-memory stages; 1 and 2
// issue tcgen05.mma for the even and the odd K blocks, each into accumulators of its own
// (waiting, issuing and committing a K block takes a warp about as long as its product); 3
// copies the factors into shared memory, eight K blocks ahead; the others, four for each
// column group, one for each quarter of the 128 TMEM lanes, drain the accumulators.
// What set this shape, measured on 128 x 256 tiles in clocks per K block (its product takes
// 512): 1900 with a release at cluster scope on the way back to the products; 1530 with each
// thread loading its own row's scale (32 lines an instruction, in the array that the products
// read their operands from); 1480 with TMEM reads, waits and additions in turn; ~1000 of them
// for a barrier of all drains around the staging of scales.
//
// Forms (one CTA per SM in each):
//   wide (large products): 128 x 256 tiles, persistent
//   narrow: 128 x 128 or 128 x 64 tiles; a cluster of S CTAs shares a tile's K blocks where there
//     are few tiles, and adds its sums up through distributed shared memory, in rank order
// Rows past M are never stored; a small M shrinks the loaded rows of x, not the product.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>

#include "layers.cuh"

namespace uno {
namespace fp8lin {

constexpr int BM = 128;
constexpr int kRowBytes = 128;       // bytes of a K block's row: one 128-byte swizzle row
constexpr int kRoles = 4;            // warps before the draining ones
constexpr int kMaxStages = 16;
constexpr int kMaxSplit = 8;         // CTAs that share a tile's K blocks
constexpr int kChunk = 8;            // K blocks whose factors are staged together
constexpr int kFactorPitch = BM + 4; // floats of a K block's row factors (writes on 32 banks)

struct Params {
    int M, N;              // rows and columns of Y
    int nk8, nk16;         // K blocks of e4m3 and of bf16
    int m_tiles;           // row tiles
    int first, tiles;      // this launch's tiles: first .. tiles - 1
    int stages;
    uint32_t a_rows;       // rows of x loaded per K block (a multiple of 8, at most 128)
    const float* xs;       // [M, nk8]
    const float* ws;       // [ceil(N / 128), nk8]
    const float* gate;     // [M], or NULL: factor 1 for the bf16 blocks
    float scale;
    void* y;
    int y_f32;
    int ahead;             // this call's next kernel may start before this one's end
    int after;             // started so: waits for the end of the one before, where T comes from
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

// R columns of this warp's 32 lanes, without waiting; tmem_wait makes them usable (it names
// them, so that no use is moved ahead of it)
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait(float (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
}
// True in one lane of a converged warp. The roles below run whole warps and issue under this
// predicate: the compiler then keeps descriptors and addresses in uniform registers, which a
// branch on the lane number denies it (a K block's four products issue in 150 clocks instead
// of 400, and a wait for a phase that is over takes 115 instead of 320).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// Arrive without release semantics: what is handed over is a TMEM accumulator whose reads
// have completed (tcgen05.wait::ld), no memory. A release at cluster scope costs more than
// a thousand clocks.
__device__ __forceinline__ void arrive_relaxed(uint64_t* bar) {
    asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// four bytes from global to shared memory, asynchronously; and this thread's arrival at an
// mbarrier once all it has copied so far is there
__device__ __forceinline__ void copy_async4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void block_sync() { asm volatile("barrier.sync.aligned 0;" ::: "memory"); }
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

// Wait for an mbarrier phase (bounded); gives up early once another role of this CTA has. On
// giving up it sets the flag and returns false.
__device__ __forceinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile int* gave_up) {
    for (uint32_t i = 0; i < kWaitLimit; i += 256) {
        if (*gave_up) return false;
        if (mbar_wait(bar, parity, 256)) return true;
    }
    *gave_up = 1;
    return false;
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* gave_up) {
    return mbar_try_wait(bar, parity) || wait_longer(bar, parity, gave_up);
}

// acc[at / 2 ..] += f * r
template <int N, int R>
__device__ __forceinline__ void add_scaled(uint64_t (&acc)[N], int at, float f, const float (&r)[R]) {
    const uint64_t ff = pair_of(f, f);
#pragma unroll
    for (int j = 0; j < R / 2; ++j)
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[at / 2 + j]) : "l"(ff), "l"(pair_of(r[2 * j], r[2 * j + 1])));
}

// ---------------------------------------------------------------------------------------
// stores: a draining thread holds columns of one row; a warp's store instruction should write
// whole lines. Eight lanes exchange 16-byte chunks (a transposition in three steps), after
// which lane j of the eight holds chunk j of each of their rows.
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void exchange(uint4 (&v)[8], int lane) {
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k & d) continue;
            uint4 give = up ? v[k] : v[k | d], got;
            got.x = __shfl_xor_sync(kFullMask, give.x, d);
            got.y = __shfl_xor_sync(kFullMask, give.y, d);
            got.z = __shfl_xor_sync(kFullMask, give.z, d);
            got.w = __shfl_xor_sync(kFullMask, give.w, d);
            if (up) v[k] = got;
            else v[k | d] = got;
        }
    }
}

// CW columns from `col` on of rows row0 + lane (this warp's 32 rows)
template <int CW>
__device__ __forceinline__ void store_rows(const Params& p, int row0, int col, int lane,
                                           const uint64_t (&acc)[CW / 2]) {
    if (!p.y_f32 && p.N % 8 == 0) {  // rows of bf16 that start on 16 bytes: by whole lines
        constexpr int K = CW / 8;    // chunks of 8 columns: eight, or four
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k < K) {
                const float2 a = two(acc[4 * k % (CW / 2)]), b = two(acc[(4 * k + 1) % (CW / 2)]),
                             c = two(acc[(4 * k + 2) % (CW / 2)]), d = two(acc[(4 * k + 3) % (CW / 2)]);
                v[k] = make_uint4(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y), pack_bf16(c.x, c.y), pack_bf16(d.x, d.y));
            } else {
                v[k] = make_uint4(0, 0, 0, 0);
            }
        }
        exchange(v, lane);
        const int j = lane & 7, r0 = row0 + (lane & ~7), c0 = col + 8 * j;
        const bool in = j < K && c0 < p.N;
        char* y = static_cast<char*>(p.y) + ((int64_t)r0 * p.N + c0) * 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (in && r0 + i < p.M) *reinterpret_cast<uint4*>(y) = v[i];
            y += (int64_t)p.N * 2;
        }
    } else {
        const int row = row0 + lane, n = row < p.M ? p.N - col : 0;  // columns of this row that exist
        const int64_t o = (int64_t)row * p.N + col;
        float* yf = static_cast<float*>(p.y) + o;
        __nv_bfloat16* yb = static_cast<__nv_bfloat16*>(p.y) + o;
#pragma unroll
        for (int j = 0; j < CW; j += 4) {
            const float2 a = two(acc[j / 2]), b = two(acc[j / 2 + 1]);
            if (p.y_f32 && p.N % 4 == 0) {
                if (j < n) *reinterpret_cast<float4*>(yf + j) = make_float4(a.x, a.y, b.x, b.y);
            } else if (p.y_f32) {
                if (j < n) yf[j] = a.x;
                if (j + 1 < n) yf[j + 1] = a.y;
                if (j + 2 < n) yf[j + 2] = b.x;
                if (j + 3 < n) yf[j + 3] = b.y;
            } else {
                if (j < n) yb[j] = __float2bfloat16_rn(a.x);
                if (j + 1 < n) yb[j + 1] = __float2bfloat16_rn(a.y);
                if (j + 2 < n) yb[j + 2] = __float2bfloat16_rn(b.x);
                if (j + 3 < n) yb[j + 3] = __float2bfloat16_rn(b.y);
            }
        }
    }
}

// four columns of a row
__device__ __forceinline__ void store4(const Params& p, int64_t row, int col, const float4& v) {
    const int64_t o = row * p.N + col;
    const float w[4] = {v.x, v.y, v.z, v.w};
    if (p.y_f32) {
        float* y = static_cast<float*>(p.y) + o;
        if (p.N % 4 == 0) {
            *reinterpret_cast<float4*>(y) = v;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < p.N) y[j] = w[j];
        }
    } else {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + o;
        if (p.N % 4 == 0) {
            *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < p.N) y[j] = __float2bfloat16_rn(w[j]);
        }
    }
}

// ---------------------------------------------------------------------------------------
// BN: columns of a tile; EW: draining warps. One CTA per SM: that is all the runtime's occupancy
// query allows this kernel, whatever its size. (Forms of half an SM, two of whose CTAs the
// hardware did place on one, failed with "unspecified launch failure" once in some thousand
// calls, on an SM that held two.) NB accumulators of BN columns share the SM's TMEM. The narrow
// forms drain with eight warps, whose registers need no split: sixteen took 125 us against 115
// for M 64, 4096 -> 151936, and 17.0 against 16.0 for M 512, 4096 -> 4096.
// ---------------------------------------------------------------------------------------
template <int BN, int EW>
struct Form {
    static constexpr int bn = BN, threads = 32 * (kRoles + EW);
    static constexpr int CW = BN * 4 / EW;          // columns of a draining warp
    static constexpr int C = 16;                    // columns read ahead: CW / C is even
    static constexpr int tmem = 512, NB = tmem / BN;
    static constexpr int halves = BN > kBlockCols ? BN / kBlockCols : 1;  // blocks of weight rows
    // registers a thread at launch, and after the split: the role warps give up theirs. The
    // split's sum may not exceed the launch's total.
    static constexpr bool split = BN == 256;
    static constexpr int regs = 96, role_regs = 32, drain_regs = 112;
    static_assert(!split || 32 * kRoles * role_regs + 32 * EW * drain_regs <= threads * regs, "register split");
    static constexpr int factor_bytes = 2 * kChunk * (kFactorPitch + halves) * 4;
    // dynamic shared memory: the SM's 227 KB without the static part
    static constexpr int smem = 226 * 1024 - factor_bytes - 768;
};
using Wide = Form<256, 16>;
using Narrow128 = Form<128, 8>;
using Narrow64 = Form<64, 8>;

template <class F>
__global__ void __launch_bounds__(F::threads, 1)
linear_kernel(const __grid_constant__ CUtensorMap tX, const __grid_constant__ CUtensorMap tW,
              const __grid_constant__ CUtensorMap tT, const __grid_constant__ CUtensorMap tB, const Params p) {
    constexpr int BN = F::bn, CW = F::CW, C = F::C, NB = F::NB, EW = F::threads / 32 - kRoles;
    constexpr int PITCH = BN + 4;  // floats of a row of sums in shared memory (no bank conflicts)
    extern __shared__ unsigned char dyn[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], tfull[NB], tempty[NB], sfull[2], sempty[2],
        drain[2];
    __shared__ struct {
        float x[2][kChunk][kFactorPitch];  // row factors
        float w[2][F::halves][kChunk];     // column factors
    } scales;
    __shared__ uint32_t tmem_base;
    __shared__ int s_gave_up;

    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t ST = (uint32_t)p.stages;
    const uint32_t a_bytes = p.a_rows * kRowBytes;
    constexpr uint32_t b_bytes = BN * kRowBytes;
    const uint32_t ring_b = ring + ST * a_bytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* gave_up = &s_gave_up;
    const uint32_t S = F::bn == 256 ? 1u : cluster_size(), rank = F::bn == 256 ? 0u : cluster_rank();
    const int tile0 = p.first + blockIdx.x / S, step = gridDim.x / S;
    // this CTA's share of the K blocks of its tiles
    const int nk = p.nk8 + p.nk16;
    const int kb0 = (int)((int64_t)nk * rank / S), kb1 = (int)((int64_t)nk * (rank + 1) / S);

    // draining warps that take part: with a single row tile, those whose rows exist (the others,
    // polling barriers for nothing, took a third of the speed of a call of a few rows)
    const int live = p.m_tiles == 1 ? EW / 4 * ((p.M + 31) / 32) : EW;
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], live);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sfull[b], 64);  // a lane's copies, and its stores
            mbar_init(&sempty[b], live);
            mbar_init(&drain[b], 1);
        }
        s_gave_up = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "n"(F::tmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base;
    // this call's next kernel may start on the SMs that this one of few CTAs leaves free (before it
    // reads T, and before it ends, it waits for this grid's end)
    if (p.ahead) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp < kRoles) {
    if (F::split) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F::role_regs));
    if (warp == 0) {
        const bool one = elect_one();
        uint32_t s = 0, ph = 1, got = 0;
        bool waited = !p.after, ok = true;  // (a lane that has given up keeps the others company)
        for (int tile = tile0; tile < p.tiles; tile += step) {
            const int m0 = (tile % p.m_tiles) * BM, n0 = (tile / p.m_tiles) * BN;
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = ok && (got < ST || wait_phase(&empty[s], ph, gave_up));
                __syncwarp();  // (what is issued may end the next phase: a lane still polling would miss its own)
                const bool low = kb >= p.nk8;
                if (low && !waited) {
                    asm volatile("griddepcontrol.wait;\n\tfence.proxy.async.global;" ::: "memory");
                    waited = true;
                }
                if (one && ok) {
                    mbar_arrive_expect_tx(&full[s], a_bytes + b_bytes);
                    const uint32_t a = ring + s * a_bytes, b = ring_b + s * b_bytes;
                    if (low) {
                        load_2d(a, &tT, (kb - p.nk8) * 64, m0, &full[s]);
                        load_2d(b, &tB, (kb - p.nk8) * 64, n0, &full[s]);
                    } else {
                        load_2d(a, &tX, kb * 128, m0, &full[s]);
                        load_2d(b, &tW, kb * 128, n0, &full[s]);
                    }
                }
                __syncwarp();
                got += ok;
                if (++s == ST) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // (what follows on the stream waits for this grid only)
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
        // Nothing may still be on its way to this CTA's shared memory when it ends: the last commits
        // arrive at `empty` on their own, after the accumulators they follow have been seen (an
        // arrival at the barriers of the next CTA in this place would break its ring). Loads that
        // no product will read: let them land.
        for (uint32_t j = got > ST ? got - ST : 0; j < got; ++j) {
            if (*gave_up) mbar_wait(&full[j % ST], (j / ST) & 1, 1u << 16);
            else wait_phase(&empty[j % ST], (j / ST) & 1, gave_up);
        }
        __syncwarp();
    } else if (warp <= 2) {
        // K block i of the CTA goes to accumulator i mod NB (NB is even)
        const bool one = elect_one();
        const uint64_t da0 = operand_desc(ring), db0 = operand_desc(ring_b);
        const uint32_t odd = (uint32_t)warp - 1u, nkl = (uint32_t)(kb1 - kb0);
        const uint32_t mine = p.tiles > tile0 ? (uint32_t)((p.tiles - 1 - tile0) / step + 1) : 0u;
        uint32_t b = odd, bph = 1, s = odd % ST, ph = (odd / ST) & 1u;
        uint32_t kl = nkl ? odd % nkl : 0;
        bool ok = true;
        for (uint32_t i = odd; i < mine * nkl; i += 2) {
            // (the two first polls are in flight together)
            const bool free = i < (uint32_t)NB || mbar_try_wait(&tempty[b], bph);
            ok = ok && wait_phase(&full[s], ph, gave_up) && (free || wait_longer(&tempty[b], bph, gave_up));
            __syncwarp();  // (what is issued may end the next phases: a lane still polling would miss its own)
            fence_after();
            if (one && ok) {
                const uint64_t da = da0 + (uint64_t)((s * a_bytes) >> 4), db = db0 + (uint64_t)((s * b_bytes) >> 4);
                const uint32_t d = tmem + b * BN;
                if (kb0 + (int)kl < p.nk8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 32 bytes of K per instruction
                        mma_e4m3(d, da + 2 * k, db + 2 * k, idesc_e4m3(BM, BN), k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_bf16(d, da + 2 * k, db + 2 * k, idesc_bf16(BM, BN), k > 0);
                }
                commit(&tfull[b]);
                commit(&empty[s]);
            }
            __syncwarp();
            s += 2;
            if (s >= ST) {
                s -= ST;
                ph ^= 1u;
            }
            b += 2;
            if (b >= (uint32_t)NB) {
                b -= NB;
                bph ^= 1u;
            }
            for (kl += 2; kl >= nkl;) kl -= nkl;
        }
        if (*gave_up) {  // products in flight end before their memory is given back
            if (one) commit(&drain[odd]);
            mbar_wait(&drain[odd], 0, 1u << 16);
        }
        __syncwarp();
    } else {
        // The scales of the next eight K blocks, copied without passing through registers: a row's
        // eight are one 32-byte sector. (Through registers, four loads a lane at a time, this warp
        // held up everything: 700 clocks a K block.) For the adapter's K blocks the row's factor is
        // its gate, the column's the adapter's scale.
        uint32_t cb = 0, ph = 1, chunks = 0;
        bool ok = true;
        for (int tile = tile0; tile < p.tiles; tile += step) {
            const int m0 = (tile % p.m_tiles) * BM, n0 = (tile / p.m_tiles) * BN;
            for (int kc = kb0; kc < kb1; kc += kChunk, ++chunks) {
                // this lane's K block kb = kc + lane % 8, rows lane / 8, + 4, + 8, ...
                const int k = lane & (kChunk - 1), kb = kc + k, row = m0 + lane / kChunk;
                const bool low = kb >= p.nk8;
                const float* src = low ? p.gate : p.xs;
                const int step_row = low ? 1 : p.nk8;
                if (src) src += low ? row : (int64_t)row * p.nk8 + kb;
                ok = ok && (chunks < 2 || wait_phase(&sempty[cb], ph, gave_up));
                if (ok) {
                    float* x = &scales.x[cb][k][lane / kChunk];
                    const int rows = kb < kb1 ? p.M - row : 0;
                    if (src) {
#pragma unroll 8
                        for (int r = 0; r < BM; r += 4)
                            if (r < rows) copy_async4(x + r, src + (int64_t)r * step_row);
                    } else {
                        for (int r = 0; r < BM; r += 4) x[r] = 1.f;
                    }
                    if (lane < F::halves * kChunk) {
                        const int n = n0 + (lane / kChunk) * kBlockCols;
                        float* w = &scales.w[cb][lane / kChunk][k];
                        if (low) *w = p.gate ? p.scale : 1.f;
                        else if (n < p.N && kb < kb1) copy_async4(w, p.ws + (int64_t)(n / kBlockCols) * p.nk8 + kb);
                    }
                    arrive_after_copies(&sfull[cb]);
                    mbar_arrive(&sfull[cb]);
                }
                cb ^= 1u;
                if (cb == 0) ph ^= 1u;
            }
            __syncwarp();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    }
    // (each side of the register split runs to its end by itself: nothing behind a join is
    // compiled for the larger share and run by a warp of the smaller)
    if (S > 1) {
        cluster_sync();  // (the sums are laid down)
        cluster_sync();  // no CTA leaves while another reads its sums
    }
    fence_before();
    block_sync();
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(F::tmem) : "memory");
    if (threadIdx.x == 0 && *gave_up) record_device_status(p.status, (uint32_t)UNO_ERR_TIMEOUT);
    } else {
        if (F::split) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F::drain_regs));
        // ---- draining: acc += factor * accumulator, one row a thread, CW columns. C columns are
        // read ahead of those being added up, across K blocks too. ----
        const int quarter = warp & 3, group = (warp - kRoles) >> 2, r0 = quarter * 32;
        const uint32_t taddr = tmem + (uint32_t)(group * CW) + ((uint32_t)r0 << 16);
        const int half = F::halves > 1 ? group * CW / kBlockCols : 0;
        uint32_t b = 0, bph = 0, cb = 0, sph = 0;
        uint64_t acc[CW / 2];  // (column pairs of one row)
        // A wait that gives up sets the flag, and the loops run on to their end: what they add up
        // then is not stored.
        auto next_block = [&](int k) {  // accumulator and factor of the CTA's K block k after this one
            if (lane == 0) arrive_relaxed(&tempty[b]);
            if (++b == (uint32_t)NB) {
                b = 0;
                bph ^= 1u;
            }
            if ((k & (kChunk - 1)) == 0 || kb0 + k == kb1) {  // the chunk of factors is used up
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty[cb]);
                cb ^= 1u;
                if (cb == 0) sph ^= 1u;
            }
        };
        for (int tile = tile0; tile < p.tiles; tile += step) {
            const int m0 = (tile % p.m_tiles) * BM, col = (tile / p.m_tiles) * BN + group * CW;
            if (p.m_tiles == 1 && r0 >= p.M) break;  // (not among the live ones)
            if (m0 + r0 >= p.M) {  // rows past M in the last row tile: only keep the barriers going
                for (int k = 0; k < kb1 - kb0; ++k) {
                    if ((k & (kChunk - 1)) == 0) wait_phase(&sfull[cb], sph, gave_up);
                    wait_phase(&tfull[b], bph, gave_up);
                    __syncwarp();
                    next_block(k + 1);
                }
                continue;
            }
#pragma unroll
            for (int j = 0; j < CW / 2; ++j) acc[j] = 0;
            float r[2][C];
            wait_phase(&sfull[cb], sph, gave_up);
            float f = scales.x[cb][0][r0 + lane] * scales.w[cb][half][0];
            wait_phase(&tfull[b], bph, gave_up);
            fence_after();
            __syncwarp();
            tmem_load(taddr + b * BN, r[0]);
            for (int k = 0; k < kb1 - kb0; ++k) {
                const float fk = f;
#pragma unroll
                for (int c = 0; c < CW; c += C) {
                    tmem_wait(r[c / C & 1]);
                    if (c + C < CW) {
                        tmem_load(taddr + b * BN + (uint32_t)(c + C), r[c / C + 1 & 1]);
                    } else {
                        // this accumulator is read and may be filled again; on to the next one
                        fence_before();
                        next_block(k + 1);
                        if (kb0 + k + 1 < kb1) {
                            if (((k + 1) & (kChunk - 1)) == 0) wait_phase(&sfull[cb], sph, gave_up);
                            const int kn = (k + 1) & (kChunk - 1);
                            const float xs = scales.x[cb][kn][r0 + lane], ws = scales.w[cb][half][kn];
                            wait_phase(&tfull[b], bph, gave_up);
                            f = xs * ws;
                            fence_after();
                            __syncwarp();
                            tmem_load(taddr + b * BN, r[c / C + 1 & 1]);
                        }
                    }
                    if (kb0 + k < p.nk8) {
                        add_scaled(acc, c, fk, r[c / C & 1]);
                    } else {
                        if (fk != 0.f) add_scaled(acc, c, fk, r[c / C & 1]);  // no adapter on a row whose factor is 0
                        __syncwarp();
                    }
                }
            }
            if (S == 1 && *gave_up == 0) store_rows<CW>(p, m0 + r0, col, lane, acc);
        }
        if (S > 1) {
            // ---- the CTAs' sums through shared memory (the ring: this CTA's products, which this
            // warp has seen end, were its last readers) ----
            const int m0 = (tile0 % p.m_tiles) * BM, n0 = (tile0 / p.m_tiles) * BN;
            const int rows = p.M - m0 < BM ? p.M - m0 : BM;
            if (r0 + lane < rows) {
                const uint32_t at = ring + (uint32_t)((r0 + lane) * PITCH + group * CW) * 4u;
#pragma unroll
                for (int j = 0; j < CW / 2; j += 2)
                    asm volatile("st.shared.v2.b64 [%0], {%1,%2};" ::"r"(at + j * 8u), "l"(acc[j]), "l"(acc[j + 1])
                                 : "memory");
            }
            __syncwarp();
            cluster_sync();
            // rank r of the cluster writes its share of the rows, four columns a thread
            const int first = (int)(rows * rank / S), n = ((int)(rows * (rank + 1) / S) - first) * (BN / 4);
            for (int i = threadIdx.x - 32 * kRoles; i < n && *gave_up == 0; i += 32 * EW) {
                const int r = first + i / (BN / 4), c = (i % (BN / 4)) * 4;
                if (n0 + c >= p.N) continue;
                const uint32_t at = ring + (uint32_t)(r * PITCH + c) * 4u;
                float4 part[kMaxSplit];
#pragma unroll
                for (uint32_t k = 0; k < kMaxSplit; ++k)
                    part[k] = k < S ? ld_cluster(at, k) : make_float4(0.f, 0.f, 0.f, 0.f);
                float4 v = part[0];
#pragma unroll
                for (uint32_t k = 1; k < kMaxSplit; ++k)
                    v.x += part[k].x, v.y += part[k].y, v.z += part[k].z, v.w += part[k].w;
                store4(p, m0 + r, n0 + c, v);
            }
            __syncwarp();
            cluster_sync();  // no CTA leaves while another reads its sums
        }
        __syncwarp();
        fence_before();
        block_sync();
    }
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

// How a product of M x N with nk K blocks is run
struct Shape {
    int BN;      // 256: the wide form
    int S;       // CTAs per tile
    int stages;
    uint32_t a_rows;
};

// A turn of wide tiles takes as long as 8 / 5 turns of narrow ones. M 256, 2560 -> 9728, rank 64:
// one turn of wide tiles 18.7 us, two of narrow ones 22.4. M 512, 4096 -> 4096: one of each, 21.3
// against 16.0.
constexpr int kWideCost = 8, kNarrowCost = 5;

template <class F>
Shape shape_of(int64_t M, int S) {
    Shape c{};
    c.BN = F::bn;
    c.S = S;
    c.a_rows = M >= BM ? BM : (uint32_t)((M + 7) / 8 * 8);
    const size_t stage = (size_t)(c.a_rows + F::bn) * kRowBytes;
    c.stages = (int)((F::smem - 1024) / stage);
    if (c.stages > kMaxStages) c.stages = kMaxStages;
    // (A launch takes all of the SM's shared memory, whatever the ring needs: no other CTA with TMEM
    // of its own, this kernel's or another's, fits beside. The products read 128 rows of x from
    // every stage, loaded or not, and a cluster's sums lie over the ring: both end inside it.)
    static_assert(F::smem >= 1024 + BM * (F::bn + 4) * 4 || F::bn == 256, "a cluster's sums");
    return c;
}

// What a form needs to know of the current device, found at its first call there: its kernel's
// attributes are set, its registers checked, and the clusters of 2, 4 and 8 CTAs counted that
// run at once (GPCs of uneven size hold fewer than SMs / S).
struct Facts {
    int clusters[4];  // of 1 << i CTAs
};
template <class F>
uno_status facts_of(int sms, Facts& f) {
    static std::atomic<uint64_t> known[kDevices];  // 16 bits each for 1, 2, 4 and 8 CTAs; 0: not yet
    int dev = 0;
    uno_status s = check_cuda(cudaGetDevice(&dev), "cudaGetDevice");
    if (s != UNO_OK) return s;
    uint64_t k = dev < kDevices ? known[dev].load(std::memory_order_acquire) : 0;
    if (!k) {
        s = check_cuda(cudaFuncSetAttribute(linear_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::smem),
                       "cudaFuncSetAttribute(fp8 linear)");
        cudaFuncAttributes a;
        if (s == UNO_OK)
            s = check_cuda(cudaFuncGetAttributes(&a, linear_kernel<F>), "cudaFuncGetAttributes(fp8 linear)");
        if (s != UNO_OK) return s;
        // the kernel's register split waits for what the launch did not bring
        if (F::split && a.numRegs < F::regs)
            return set_error(UNO_ERR_CUDA, "fp8 linear was built with %d registers a thread, %d are needed", a.numRegs,
                             F::regs);
        k = (uint64_t)sms;
        for (int i = 1; i < 4 && F::bn != Wide::bn; ++i) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 1u << i;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.blockDim = dim3((unsigned)F::threads);
            cfg.gridDim = dim3((unsigned)sms & ~7u);
            cfg.dynamicSmemBytes = F::smem;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int n = 0;
            s = check_cuda(cudaOccupancyMaxActiveClusters(&n, linear_kernel<F>, &cfg),
                           "cudaOccupancyMaxActiveClusters");
            if (s != UNO_OK) return s;
            k |= (uint64_t)(n < 0xFFFF ? n : 0xFFFF) << (16 * i);
        }
        if (dev < kDevices) known[dev].store(k, std::memory_order_release);
    }
    for (int i = 0; i < 4; ++i) f.clusters[i] = (int)(k >> (16 * i) & 0xFFFF);
    return UNO_OK;
}

// The narrow form F of a product: CTAs per tile, and the K blocks that a CTA takes in turn (what
// such a call's time goes by). `beside` CTAs of the kernel before may still hold SMs, and a cluster
// that finds no place waits for them all: where they are few, clusters are counted without them.
template <class F>
uno_status narrow_shape(int64_t M, int64_t N, int nk, int sms, int beside, Shape& c, int64_t& in_turn) {
    Facts f;
    const uno_status s = facts_of<F>(sms, f);
    if (s != UNO_OK) return s;
    const int64_t tiles = (M + BM - 1) / BM * ((N + F::bn - 1) / F::bn);
    if (beside * 4 <= sms)
        for (int& n : f.clusters) n = n * (sms - beside) / sms;
    int i = 0;
    while (i < 3 && tiles <= f.clusters[i + 1] && nk >= 4 << i) ++i;
    in_turn = (tiles + sms - 1) / sms * ((nk + (1 << i) - 1) >> i);
    if (i > 0) in_turn = (nk + (1 << i) - 1) >> i;
    c = shape_of<F>(M, 1 << i);
    return UNO_OK;
}

uno_status choose(int64_t M, int64_t N, int nk, int sms, int beside, Shape& c) {
    const int64_t m_tiles = (M + BM - 1) / BM;
    auto turns = [&](int bn) { return (m_tiles * ((N + bn - 1) / bn) + sms - 1) / sms; };
    if (M > 64 && turns(Narrow128::bn) * kNarrowCost > turns(Wide::bn) * kWideCost) {
        Facts f;
        c = shape_of<Wide>(M, 1);
        return facts_of<Wide>(sms, f);
    }
    // The form with fewer K blocks in turn; M 16, 4096 -> 4096 from L2: 8 with 128 columns and clusters
    // of four, 8.3 us, 16 with 64 columns and clusters of two, 10.9. Where both have as many, the one
    // whose block is shorter: M 37, 4992 -> 700: 64 columns 6.9 us, 128 columns 7.4.
    Shape c64;
    int64_t in_turn, in_turn64;
    uno_status s = narrow_shape<Narrow128>(M, N, nk, sms, beside, c, in_turn);
    if (s == UNO_OK) s = narrow_shape<Narrow64>(M, N, nk, sms, beside, c64, in_turn64);
    if (s == UNO_OK && in_turn64 <= in_turn) c = c64;
    return s;
}

template <class F>
uno_status launch(const Shape& c, const CUtensorMap (&maps)[4], const Params& p, int sms, cudaStream_t stream) {
    // persistent, except where a cluster shares a tile
    const int64_t tiles = p.tiles - p.first, units = c.S > 1 || tiles < sms ? tiles : sms;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    cfg.blockDim = dim3((unsigned)F::threads);
    cfg.gridDim = dim3((unsigned)(units * c.S));
    cfg.dynamicSmemBytes = F::smem;
    cfg.stream = stream;
    cfg.attrs = attrs;
    if (c.S > 1) {
        attrs[0].id = cudaLaunchAttributeClusterDimension;
        attrs[0].val.clusterDim.x = (unsigned)c.S;
        attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
    }
    if (p.after) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    return check_cuda(cudaLaunchKernelEx(&cfg, linear_kernel<F>, maps[0], maps[1], maps[2], maps[3], p),
                      "launch(fp8 linear)");
}

// one product: e4m3 blocks over d_in columns (or none), bf16 blocks over r columns (or none)
uno_status product(const void* xq, const void* wq, int64_t d_in, const void* t, const void* b, int64_t r, Params p,
                   cudaStream_t stream, int beside, int* ctas) {
    const int sms = device_sms();
    p.status = device_status_ptr();
    if (sms == 0 || !p.status) return set_error(UNO_ERR_CUDA, "the current device's properties cannot be read");
    p.nk8 = (int)((d_in + 127) / 128);
    p.nk16 = (int)((r + 63) / 64);
    Shape c;
    uno_status s = choose(p.M, p.N, p.nk8 + p.nk16, sms, beside, c);
    if (s != UNO_OK) return s;
    p.m_tiles = (p.M + BM - 1) / BM;
    const int nk = p.nk8 + p.nk16;
    const int64_t tiles = (int64_t)p.m_tiles * ((p.N + c.BN - 1) / c.BN);
    p.tiles = (int)tiles;
    if (ctas) *ctas = (int)(c.S > 1 || tiles < sms ? tiles * c.S : sms);
    auto run = [&](const Shape& c, Params p) {
        p.stages = c.stages;
        p.a_rows = c.a_rows;
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
        return c.BN == Wide::bn        ? launch<Wide>(c, maps, p, sms, stream)
               : c.BN == Narrow128::bn ? launch<Narrow128>(c, maps, p, sms, stream)
                                       : launch<Narrow64>(c, maps, p, sms, stream);
    };
    // The persistent CTAs' last turn may hold few tiles (a head of 151936 columns has 594 of 256
    // columns for 148 SMs: four turns and two tiles). Then the last columns' tiles are shared by
    // clusters of eight in a launch of their own, and the others start beside it: M 128, 4096 ->
    // 151936 123 us in place of 132, M 8, 4096 -> 19200 (one turn) 24 in place of 28. Not with more
    // tiles (M 2000, 2048 -> 9728, 32 tiles: 68 against 60), fewer K blocks (M 16, 2560 -> 151936:
    // 75.2 against 73.9) or more turns (M 64, 4096 -> 151936, eight: 119.7 us either way).
    if (c.S == 1 && c.BN >= Narrow128::bn && tiles > sms && tiles / sms <= 4 && nk >= 32) {
        Facts f;
        s = facts_of<Narrow128>(sms, f);
        if (s != UNO_OK) return s;
        const int64_t whole = tiles / sms * sms / p.m_tiles * (c.BN / Narrow128::bn);  // columns of narrow tiles
        const int64_t rest = p.m_tiles * ((p.N + Narrow128::bn - 1) / Narrow128::bn - whole);
        if (rest > 0 && rest <= f.clusters[3]) {
            Params last = p;
            last.first = (int)(p.m_tiles * whole);
            last.tiles = (int)(last.first + rest);
            last.ahead = 1;
            s = run(shape_of<Narrow128>(p.M, 8), last);
            if (s != UNO_OK) return s;
            p.tiles = (int)(p.m_tiles * (whole / (c.BN / Narrow128::bn)));
            p.after = 1;
        }
    }
    return run(c, p);
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
        return set_error(UNO_ERR_UNSUPPORTED,
                         "d_in a multiple of 16 up to 65536, d_out and M up to 2^20 are supported");
    if (rank % 8 || rank > 256) return set_error(UNO_ERR_UNSUPPORTED, "rank must be 0 or a multiple of 8 and <= 256");
    if (rank && y_dtype == UNO_F32) return set_error(UNO_ERR_UNSUPPORTED, "float32 output is supported with rank 0");
    // tiles times K blocks: they are counted over a CTA's tiles in 32 bits
    const int64_t tiles = (M + 127) / 128 * (M > 64 ? (d_out + 255) / 256 : (d_out + 127) / 128);
    if (tiles * ((d_in + 127) / 128 + (rank + 63) / 64) > 0x7FFFFFFF)
        return set_error(UNO_ERR_UNSUPPORTED, "too many output tiles");
    if (M == 0) return UNO_OK;
    if (!x_q || !x_scale || !w_q || !w_scale || !y) return set_error(UNO_ERR_INVALID_ARG, "a tensor pointer is NULL");
    if (rank && (!x || !lora_a || !lora_b))
        return set_error(UNO_ERR_INVALID_ARG, "rank > 0 needs x, lora_a and lora_b");
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
    int beside = 0;  // CTAs that make T
    if (adapter) {   // T = bf16(X A^T)
        fp8lin::Params t = p;
        t.N = (int)rank;
        t.y = workspace;
        t.ahead = 1;
        const uno_status s = fp8lin::product(nullptr, nullptr, 0, x, lora_a, d_in, t, st, 0, &beside);
        if (s != UNO_OK) return s;
    }
    p.N = (int)d_out;
    p.xs = x_scale;
    p.ws = w_scale;
    p.gate = adapter ? row_gate : nullptr;
    p.scale = scale;
    p.y = y;
    p.y_f32 = y_dtype == UNO_F32;
    p.after = adapter;
    return fp8lin::product(x_q, w_q, d_in, workspace, lora_b, adapter ? rank : 0, p, st, beside, nullptr);
}
