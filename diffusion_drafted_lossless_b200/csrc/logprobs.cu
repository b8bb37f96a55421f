// logprobs.cu — log probabilities of given tokens, entropy, the most probable alternatives,
// and the gradient.
//
//   s = sum exp((x - ref) / T),  a = sum exp((x - ref) / T) (x - ref)    (ref: near the maximum)
//   log p_v = (x_v - max) / T - log s_max,   entropy = log s_max - a_max / (s_max T)
// where s_max, a_max are the sums moved to ref = max. exp is ex2 of (x - ref) (log2 e / T), as
// Sums below says for values and temperatures of every size.
//
// One pass over the row (bound: HBM, then the exponential unit: one ex2 an element). A row goes
// to a cluster of S CTAs, each with a run of it; a thread streams 16-byte pieces, four added up
// while the next four travel. The first eight pieces of all threads are a sample: its maximum is
// every thread's first reference, so that references move (and sums are rescaled) only where a
// value lies 64 octaves above; and the top_n-th largest of the sample's 64 group maxima is a
// value that at least top_n tokens reach, so only elements at or above it (a few hundred of a
// row) are candidates for the alternatives; after a quarter of a long run the candidates so far
// raise that bound. They are appended to a list in shared memory and ranked at the end by
// counting, value first and id second: a long list first in shares, one for each warp.
// A list that overflows (a row in ascending order, a row of equal values) is no loss: its entries
// are real tokens, so the top_n-th best of them bounds the search and the run is read again for
// what beats it, until the list holds everything. Each such reading leaves about top_n of 2048 of
// what it finds, whatever the order (600 rows of 151936 bf16 that rise to their middle and fall:
// 0.89 ms in place of 4.9 with a list of the first and latest ones; in no order: 0.065).
// Measured: 2048 rows of 166144 bf16, 40% left out, 5 alternatives: 82 us, 5.0 TB/s; 16 rows of
// 151936, 20 alternatives: 10.9 us (eight CTAs a row; ranking and joining take half). With its
// gradient, 1024 rows of 151936: 157 us, 160 in a second-long run (1880 MHz), the logits read twice
// and the gradient written once.
#include <cmath>
#include <type_traits>

#include "layers.cuh"

namespace uno {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr int kGroups = 64;     // groups of 4 lanes whose maxima bound the search
constexpr int kList = 2048;     // candidates held
constexpr int kQuick = 96;      // lists up to this long are ranked at once
constexpr int kMaxTop = 32;
constexpr int kMaxSplit = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// an exponent no lower than `least`, one of nothing; a NaN stays one
template <int least = -2000>
__device__ __forceinline__ float exponent(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"((float)least));
    return y;
}

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

// One value. (Not __ldg of a __nv_bfloat16: that is an asm statement without volatile, which
// the compiler may run ahead of the condition that keeps its address inside the row.)
template <typename T>
__device__ __forceinline__ float load_one(const T* p) {
    if constexpr (std::is_same_v<T, float>) return __ldg(p);
    else return bf16_lo(__ldg(reinterpret_cast<const unsigned short*>(p)));
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// the largest of a piece (NaN passed over)
template <typename T>
__device__ __forceinline__ float piece_max(const uint4& v) {
    if constexpr (std::is_same_v<T, float>) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        auto h = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
}

// the largest of N pieces (NaN passed over)
template <typename T, int N>
__device__ __forceinline__ float pieces_max(const uint4 (&v)[N]) {
    float m;
    if constexpr (std::is_same_v<T, float>) {
        m = piece_max<T>(v[0]);
#pragma unroll
        for (int u = 1; u < N; ++u) m = fmaxf(m, piece_max<T>(v[u]));
    } else {
        auto h = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
        __nv_bfloat162 m2 = __hmax2(__hmax2(h(v[0].x), h(v[0].y)), __hmax2(h(v[0].z), h(v[0].w)));
#pragma unroll
        for (int u = 1; u < N; ++u)
            m2 = __hmax2(m2, __hmax2(__hmax2(h(v[u].x), h(v[u].y)), __hmax2(h(v[u].z), h(v[u].w))));
        m = fmaxf(__low2float(m2), __high2float(m2));
    }
    return fmaxf(m, -INFINITY);
}

// (x - ref) / T in octaves, c4 being 4 log2 e / T: a quarter of the difference, which is always
// within float32, rounded once, and the product.
__device__ __forceinline__ float octaves(float x, float ref, float c4) { return fmaf(x, 0.25f, -0.25f * ref) * c4; }

// A thread's running sums over what it has read, in octaves: s = sum 2^arg, a = sum 2^arg arg.
// Beside an ordinary reference arg is x c - R in one rounding, R = ref c as float32 holds it.
// R is off by half a unit of its own, the same for every element, and moving to another
// reference takes that back; below 2^20 octaves it is at most a sixteenth, so no weight near the
// maximum's overflows or is lost. Values below -1e30, -inf among them, count as -1e30: with c
// between 1e-20 and 1e8 that is 1e10 octaves below any ordinary reference at least, and 1e38 at
// most, in float32's range. Beside any other reference, or with any other c, arg is
// octaves(x, ref), a subtraction and an instruction more an element.
struct Sums {
    float ref, R, max, s, a;
    bool ordinary;
};
constexpr float kLow = -1e30f, kMinC = 1.5e-20f, kMaxC = 1e8f, kMaxR = 1048576.f;

__device__ __forceinline__ void set_ref(Sums& t, float ref, float c, bool plain) {
    t.ref = ref;
    t.R = ref * c;
    t.ordinary = plain && fabsf(t.R) < kMaxR;
}

// the sums times 2^d, for a reference d octaves further up
__device__ __forceinline__ void shift(Sums& t, float d) {
    const float f = ex2(d);
    t.a = f == 0.f ? 0.f : f * fmaf(d, t.s, t.a);
    t.s *= f;
}

// how many octaves this thread's reference lies above `to`
__device__ __forceinline__ float above(const Sums& t, float to, float c, float c4) {
    return t.ordinary ? fmaf(-to, c, t.R) : octaves(t.ref, to, c4);
}

// move to another reference
__device__ __forceinline__ void move_ref(Sums& t, float to, float c, float c4, bool plain) {
    const Sums old = t;
    set_ref(t, to, c, plain);
    if (old.s == 0.f) t.a = 0.f;
    else shift(t, above(old, to, c, c4) + (t.ordinary ? fmaf(to, c, -t.R) : 0.f));  // (R's rounding)
}

__device__ __forceinline__ void add_one(Sums& t, float x, float c, float c4) {
    // (an ordinary R is finite, any other ref is finite or +inf: -inf has no weight)
    const float arg = exponent(t.ordinary ? fmaf(x, c, -t.R) : octaves(x, t.ref, c4)), e = ex2(arg);
    t.s += e;
    t.a = fmaf(e, arg, t.a);
}

// The pieces of a row beside an ordinary reference, two elements at a time.
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
template <typename T>
__device__ __forceinline__ void add_piece(const uint4& v, uint64_t minus_R, uint64_t c2, uint64_t& s2, uint64_t& a2) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    constexpr int N = 16 / (int)sizeof(T) / 2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint64_t x;
        if constexpr (std::is_same_v<T, float>) {
            float lo, hi;
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(lo) : "f"(__uint_as_float(w[2 * i])), "f"(kLow));
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(hi) : "f"(__uint_as_float(w[2 * i + 1])), "f"(kLow));
            x = pair_of(lo, hi);
        } else {
            uint32_t m;
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w[i]), "r"(0xF14AF14Au));  // -1.0002e30 twice
            x = pair_of(bf16_lo(m), bf16_hi(m));
        }
        const uint64_t arg = fma2(x, c2, minus_R);
        const uint64_t e = pair_of(ex2(two(arg).x), ex2(two(arg).y));
        s2 = add2(s2, e);
        a2 = fma2(e, arg, a2);
    }
}

// candidates found so far by this CTA, and the bound that new ones have to reach
struct Search {
    unsigned long long* list;
    unsigned int* count;
};

// Past the list's end: in the first reading its first half stays (the best of a row of equal values)
// and the second keeps the latest ones (the best of an ascending row), at no cost; when a run is read
// again, entry number `at` takes the place of one of the list with a chance of kList / (at + 1), which
// leaves an even sample of all that was found.
template <bool AGAIN = false>
__device__ __forceinline__ void append(const Search& q, float x, uint32_t id) {
    const unsigned int at = atomicAdd(q.count, 1u);
    unsigned int slot = at;
    if (at >= kList) slot = AGAIN ? __umulhi(at * 0x9E3779B1u, at + 1u) : kList / 2 + at % (kList / 2);
    if (!AGAIN || slot < kList) q.list[slot] = pack_candidate(float_key(x), id);
}

struct Args {
    int64_t V;
    float c, c4, inv_t4;       // log2 e / T, and four times that; 4 / T
    bool plain;                // c allows ordinary references
    const int32_t* tokens;
    int top_n;
    float *logprob, *entropy, *stats;
    int32_t* top_ids;
    float* top_lp;
};

__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_peer_f32(const float* p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_peer_u64(const unsigned long long* p, uint32_t rank) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(p, rank)) : "memory");
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const T* __restrict__ logits, const Args p) {
    constexpr int VE = kVec<T>;
    __shared__ unsigned long long list[kList];
    __shared__ unsigned long long best[kMaxTop];          // this run's top candidates, in order
    __shared__ unsigned long long merged[kWarps * kMaxTop];  // the warps' or the CTAs' best
    static_assert(kWarps >= kMaxSplit, "one array for both");
    __shared__ uint4 laid[kWarps][32 * kUnroll];           // pieces that hold candidates
    __shared__ float group[kGroups];
    __shared__ float part[kWarps][4];
    __shared__ float run[4];                               // this run's ref, max, s, a
    __shared__ float s_ref, s_bound;
    __shared__ unsigned int s_count;
    __shared__ unsigned long long s_kth;

    const uint32_t S = cluster_size(), rank = cluster_rank();
    const int64_t n = blockIdx.x / S;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int k = p.top_n;

    const int32_t tok = p.tokens ? p.tokens[n] : 0;
    if (tok < 0 || tok >= p.V) {  // a row that is left out (the whole cluster leaves)
        if (rank == 0) {
            if (tid == 0) {
                if (p.logprob) p.logprob[n] = 0.f;
                if (p.entropy) p.entropy[n] = 0.f;
                if (p.stats) p.stats[2 * n] = p.stats[2 * n + 1] = 0.f;
            }
            if (tid < k) {
                p.top_ids[n * k + tid] = -1;
                p.top_lp[n * k + tid] = -INFINITY;
            }
        }
        return;
    }

    const T* row = logits + n * p.V;
    // 16-byte pieces from the first aligned element on; the elements before and behind them
    // are taken one by one by the first CTA
    const int64_t mis = (int64_t)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int64_t head = mis ? (VE - mis < p.V ? VE - mis : p.V) : 0;
    const int64_t pieces = (p.V - head) / VE, tail = p.V - head - pieces * VE;
    const int64_t lo = pieces * rank / S, hi = pieces * (rank + 1) / S;
    const uint4* body = reinterpret_cast<const uint4*>(row + head);
    // edge element tid of the first CTA: id, or -1
    int64_t edge = -1;
    if (rank == 0 && tid < head) edge = tid;
    if (rank == 0 && tid >= 32 && tid - 32 < tail) edge = p.V - tail + (tid - 32);
    const float edge_x = load_one(row + (edge >= 0 ? edge : 0));

    const Search q{list, &s_count};
    const float ninf = -INFINITY;
    const uint32_t none = std::is_same_v<T, float> ? 0xFF800000u : 0xFF80FF80u;  // -inf
    // turn `it` of this thread: pieces it * kTurn + tid, + kThreads, ... of the run
    constexpr int kTurn = kUnroll * kThreads;
    const int run_pieces = (int)(hi - lo), turns = (run_pieces + kTurn - 1) / kTurn;
    const uint4* mine = body + lo + tid;
    auto load = [&](uint4(&v)[kUnroll], int it) {
        const uint4* at = mine + (int64_t)it * kTurn;
        if ((it + 1) * (int64_t)kTurn <= run_pieces) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) v[u] = ld_stream_v4(at + u * kThreads);
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                v[u] = it * (int64_t)kTurn + u * kThreads + tid < run_pieces ? ld_stream_v4(at + u * kThreads)
                                                                            : make_uint4(none, none, none, none);
        }
    };

    // ---- the sample: every thread's first eight pieces ----
    uint4 v0[kUnroll], v1[kUnroll];
    load(v0, 0);
    load(v1, 1);
    const float m = fmaxf(pieces_max<T>(v0), pieces_max<T>(v1));
    float g = m;
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(kFullMask, g, o));
    if ((lane & 3) == 0) group[tid >> 2] = g;
    if (tid == 0) {
        s_count = 0;
        s_bound = ninf;
    }
    __syncthreads();
    {
        // four threads rank a group's maximum among all (equal ones by position): the k-th bounds
        // the search
        const int mine = tid >> 2;
        const float x = group[mine];
        int r = 0;
#pragma unroll
        for (int j = 0; j < kGroups / 4; ++j) {
            const int o = (tid & 3) * (kGroups / 4) + j;
            const float y = group[o];
            r += y > x || (y == x && o < mine);
        }
        r += __shfl_xor_sync(kFullMask, r, 1);
        r += __shfl_xor_sync(kFullMask, r, 2);
        if ((tid & 3) == 0) {
            if (r == k - 1) s_bound = x;
            if (r == 0) s_ref = fmaxf(x, -3.402823466e38f);  // finite where the sample is all -inf
        }
    }
    __syncthreads();

    const float c = p.c, c4 = p.c4;
    Sums t;
    set_ref(t, s_ref, c, p.plain);
    t.max = ninf;
    t.s = t.a = 0.f;
    float bound = k > 0 ? s_bound : INFINITY;
    // (the id of the run's first element; ids are below 2^31)
    const uint32_t id0 = (uint32_t)(head + lo * VE);

    if (edge >= 0) {
        const float x = edge_x;
        if (!((x - t.ref) * c <= 64.f)) move_ref(t, fmaxf(x, t.ref), c, c4, p.plain);
        t.max = fmaxf(t.max, x);
        add_one(t, x, c, c4);
        if (x >= bound && x > ninf) append(q, x, (uint32_t)edge);
    }
    auto take = [&](const uint4(&v)[kUnroll], int it) {
        const float cm = pieces_max<T>(v);
        t.max = fmaxf(t.max, cm);
        if ((cm - t.ref) * c > 64.f) move_ref(t, cm, c, c4, p.plain);
        // lanes that hold a candidate lay their pieces down, and the warp looks at them together,
        // one element a lane
        unsigned hits = __ballot_sync(kFullMask, cm >= bound);
        if (hits) {
            if (cm >= bound) {
                uint4* at = &laid[warp][__popc(hits & ((1u << lane) - 1u)) * kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) at[u] = v[u];
            }
            __syncwarp();
            const T* at = reinterpret_cast<const T*>(&laid[warp][0]) + lane;
            // this lane's element: of piece lane / VE, its lane % VE-th
            const uint32_t id = id0 + (uint32_t)(it * kTurn + lane / VE * kThreads + warp * 32) * VE + lane % VE;
            for (; hits; hits &= hits - 1, at += kUnroll * VE) {
                if (lane < kUnroll * VE) {
                    const float x = to_float(*at);
                    if (x >= bound && x > ninf) append(q, x, id + (__ffs(hits) - 1) * VE);
                }
            }
            __syncwarp();
        }
        if (t.ordinary) {
            const uint64_t minus_R = pair_of(-t.R, -t.R), c2 = pair_of(c, c);
            uint64_t s2 = pair_of(t.s, 0.f), a2 = pair_of(t.a, 0.f);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) add_piece<T>(v[u], minus_R, c2, s2, a2);
            t.s = two(s2).x + two(s2).y;
            t.a = two(a2).x + two(a2).y;
        } else {
#pragma unroll 1
            for (int u = 0; u < kUnroll; ++u) {
                float f[VE];
                unpack<T>(u == 0 ? v[0] : u == 1 ? v[1] : u == 2 ? v[2] : v[3], f);
#pragma unroll
                for (int e = 0; e < VE; ++e) add_one(t, f[e], c, c4);
            }
        }
    };
    // a quarter of a long run bounds the search more closely than the sample did
    const int rebound = k > 0 && turns >= 8 ? turns / 4 & ~1 : -1;
    for (int it = 0; it < turns; it += 2) {
        if (it == rebound) {
            __syncthreads();
            const int held = (int)s_count;  // (above kThreads: too many for a quick look)
            if (held <= kThreads && tid < held) {
                const unsigned long long mine = list[tid];
                int r = 0;
                for (int o = 0; o < held; ++o) r += list[o] > mine;
                if (r == k - 1) s_bound = key_float(candidate_key(mine));
            }
            __syncthreads();
            bound = s_bound;
        }
        take(v0, it);
        load(v0, it + 2);
        if (it + 1 < turns) take(v1, it + 1);
        load(v1, it + 3);
    }

    // ---- this run's sums, relative to its maximum ----
    auto combine = [&](float mx) {  // the block's sums at reference mx, valid in warp 0
        if (t.s == 0.f) t.a = 0.f;
        else shift(t, above(t, mx, c, c4));
        const float s = warp_sum(t.s), a = warp_sum(t.a);
        if (lane == 0) part[warp][1] = s, part[warp][2] = a;
    };
    const float wm = warp_max(t.max);
    if (lane == 0) part[warp][0] = wm;
    __syncthreads();
    const float mx = warp_max(part[lane & (kWarps - 1)][0]);
    combine(mx);
    __syncthreads();
    if (warp == 0) {
        const float s = warp_sum(lane < kWarps ? part[lane][1] : 0.f);
        const float a = warp_sum(lane < kWarps ? part[lane][2] : 0.f);
        if (lane == 0) run[0] = run[1] = mx, run[2] = s, run[3] = a;
    }

    // ---- this run's best k ----
    if (k > 0) {
        for (;;) {
            const unsigned int found = s_count;
            const int held = (int)(found < kList ? found : kList);
            if (tid < k) best[tid] = 0;
            if (held <= kQuick) {
                __syncthreads();
                if (tid < held) {
                    const unsigned long long mine = list[tid];
                    int r = 0;
                    for (int o = 0; o < held; ++o) r += list[o] > mine;
                    if (r < k) best[r] = mine;
                }
                __syncthreads();
                break;
            }
            // each warp's share of the list (all entries differ: ids do), then the shares' best
            const int from = held * warp / kWarps, to = held * (warp + 1) / kWarps;
            merged[tid] = 0;
            __syncwarp();  // (a warp's 32 places are its own)
            for (int j = from + lane; j < to; j += 32) {
                const unsigned long long mine = list[j];
                int r = 0;
                for (int o = from; o < to && r < k; ++o) r += list[o] > mine;
                if (r < k) merged[warp * kMaxTop + r] = mine;
            }
            __syncthreads();
            const unsigned long long mine = merged[tid];
            if (mine) {
                // (each share's best are in order: how many of them are above, by bisection)
                int r = 0;
#pragma unroll 2
                for (int w = 0; w < kWarps; ++w) {
                    int n = 0;
#pragma unroll
                    for (int half = kMaxTop / 2; half > 0; half >>= 1)
                        if (merged[w * kMaxTop + n + half - 1] > mine) n += half;
                    r += n + (merged[w * kMaxTop + n] > mine);
                }
                if (r < k) best[r] = mine;
                if (r == k - 1) s_kth = mine;
            }
            if (found <= kList) {
                __syncthreads();
                break;
            }
            // more were found than are held: read the run again for what beats the k-th held
            __syncthreads();
            const unsigned long long kth = s_kth;
            if (tid == 0) s_count = 0;
            __syncthreads();
            auto again = [&](float x, uint32_t id) {
                if (x > ninf && pack_candidate(float_key(x), id) >= kth) append<true>(q, x, id);
            };
            if (edge >= 0) again(edge_x, (uint32_t)edge);
            for (int64_t i = lo + tid; i < hi; i += kThreads) {
                const uint4 w = __ldg(body + i);
                float f[VE];
                unpack<T>(w, f);
#pragma unroll
                for (int e = 0; e < VE; ++e) again(f[e], (uint32_t)(head + i * VE + e));
            }
            __syncthreads();
        }
    } else {
        __syncthreads();
    }

    // ---- the runs of a cluster, joined by its first CTA ----
    __syncwarp();
    if (S > 1) {
        cluster_sync();
        if (rank == 0) {
            if (tid < (int)S * k) merged[tid] = ld_peer_u64(&best[tid % k], tid / k);
            if (warp == kWarps - 1) {
                const bool in = lane < (int)S;
                Sums r{};
                r.max = ninf;
                if (in) {
                    r.max = ld_peer_f32(&run[1], lane);
                    r.s = ld_peer_f32(&run[2], lane);
                    r.a = ld_peer_f32(&run[3], lane);
                }
                const float all = warp_max(r.max);
                if (r.s != 0.f) shift(r, octaves(r.max, all, c4));
                const float s = warp_sum(r.s), a = warp_sum(r.a);
                __syncwarp();
                if (lane == 0) part[0][0] = all, part[0][1] = s, part[0][2] = a;
            }
        }
        __syncthreads();
        __syncwarp();
        cluster_sync();
        if (rank != 0) return;
        if (tid < k) best[tid] = 0;
        __syncthreads();
        if (tid < (int)S * k && merged[tid]) {
            int r = 0;
            for (int o = 0; o < (int)S * k; ++o) r += merged[o] > merged[tid];
            if (r < k) best[r] = merged[tid];
        }
    } else if (tid == 0) {
        part[0][0] = run[1], part[0][1] = run[2], part[0][2] = run[3];
    }
    __syncthreads();
    const float top = part[0][0], s = part[0][1], a = part[0][2];
    const bool empty = top == ninf && s == 0.f;  // nothing can be produced
    // (s has the maximum's own weight in it, 1: what falls below it are roundings, and no log
    // probability is above 0, no entropy below; a NaN stays)
    const float sure = s < 1.f ? 1.f : s, logs = empty ? 0.f : logf(sure);
    auto nats = [&](float x) { return octaves(x, top, p.inv_t4); };  // (x - max) / T
    if (tid == 0) {
        if (p.logprob) {
            const float x = load_one(row + tok);
            p.logprob[n] = empty ? ninf : nats(x) - logs;
        }
        if (p.entropy) {
            const float h = empty ? 0.f : fmaf(-kLn2, a / sure, logs);
            p.entropy[n] = h < 0.f ? 0.f : h;
        }
        if (p.stats) {
            p.stats[2 * n] = top;
            p.stats[2 * n + 1] = logs;
        }
    }
    if (tid < k) {
        const unsigned long long b = best[tid];
        p.top_ids[n * k + tid] = b ? (int32_t)candidate_id(b) : -1;
        p.top_lp[n * k + tid] = b ? nats(key_float(candidate_key(b))) - logs : ninf;
    }
}

// ---------------------------------------------------------------------------------------
// gradient: elementwise from the row's statistics. A CTA takes kGradPieces x 256 pieces of a
// row, so the row's facts are read once for them.
// ---------------------------------------------------------------------------------------
constexpr int kGradThreads = 256, kGradPieces = 4;

struct GradArgs {
    int64_t V;
    float c4, inv_t4;  // 4 log2 e / T, 4 / T
    const int32_t* tokens;
    const float *stats, *entropy, *g_lp, *g_ent;
    int chunks;  // CTAs per row
};

// (logits may be grad itself: no restrict and no read-only loads. A thread reads its pieces
// before it writes them.)
template <typename T>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const T* logits, T* grad, const GradArgs p) {
    constexpr int VE = kVec<T>;
    const int64_t n = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x - n * p.chunks), tid = threadIdx.x;
    const T* row = logits + n * p.V;
    T* out = grad + n * p.V;
    const int32_t tok = p.tokens ? p.tokens[n] : 0;
    const float max = p.stats[2 * n], logs = p.stats[2 * n + 1];
    const bool zero = tok < 0 || tok >= p.V || max == -INFINITY;
    const float gl = !zero && p.g_lp ? 0.25f * p.g_lp[n] * p.inv_t4 : 0.f;
    const float ge = !zero && p.g_ent ? 0.25f * p.g_ent[n] * p.inv_t4 : 0.f;
    const float h = !zero && p.g_ent ? p.entropy[n] : 0.f;
    // d = -p (gl + ge (log p + h)) = p (base + slope arg), arg = log2 p
    const float l2 = logs * kLog2e, max4 = -0.25f * max, base = -fmaf(ge, h, gl), slope = -ge * kLn2;
    auto one = [&](float x, int64_t id) {
        // (from -150 on the weight is 0, whatever its factor is: that stays inside float32)
        const float arg = exponent<-150>(fmaf(fmaf(x, 0.25f, max4), p.c4, -l2));
        float d = ex2(arg) * fmaf(slope, arg, base);
        if (id == tok) d += gl;
        return zero ? 0.f : d;
    };
    auto put = [&](int64_t id, float d) {
        if constexpr (std::is_same_v<T, float>) out[id] = d;
        else out[id] = __float2bfloat16_rn(d);
    };
    auto get = [&](int64_t id) -> float {
        if constexpr (std::is_same_v<T, float>) return row[id];
        else return __bfloat162float(row[id]);
    };
    const int64_t mis = (int64_t)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int64_t head = mis ? (VE - mis < p.V ? VE - mis : p.V) : 0;
    // (rows of grad are as aligned as those of logits: both tensors start on 16 bytes)
    const int64_t pieces = (p.V - head) / VE, tail = p.V - head - pieces * VE;
    if (chunk == 0) {
        int64_t id = -1;
        if (tid < head) id = tid;
        if (tid >= 32 && tid - 32 < tail) id = p.V - tail + (tid - 32);
        if (id >= 0) put(id, one(get(id), id));
    }
    const uint4* src = reinterpret_cast<const uint4*>(row + head);
    uint4* dst = reinterpret_cast<uint4*>(out + head);
    const int64_t i0 = (int64_t)chunk * (kGradThreads * kGradPieces) + tid;
    uint4 v[kGradPieces];
#pragma unroll
    for (int u = 0; u < kGradPieces; ++u) {
        const int64_t i = i0 + u * kGradThreads;
        v[u] = i < pieces && !zero ? src[i] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kGradPieces; ++u) {
        const int64_t i = i0 + u * kGradThreads;
        if (i >= pieces) continue;
        float f[VE];
        unpack<T>(v[u], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = one(f[e], head + i * VE + e);
        if constexpr (std::is_same_v<T, float>)
            dst[i] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                __float_as_uint(f[3]));
        else
            dst[i] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                pack_bf16(f[6], f[7]));
    }
}

template <typename T>
uno_status logprobs_launch(const void* logits, int64_t N, const Args& p, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms == 0) return set_error(UNO_ERR_CUDA, "the current device's properties cannot be read");
    // CTAs per row: as many as fill the GPU twice, while each still has a few turns of work
    int S = 1;
    while (S < kMaxSplit && N * S * 2 <= 2 * (int64_t)sms && p.V >= (int64_t)S * 2 * kThreads * kVec<T>) S *= 2;
    if (N * S > 0x7FFFFFFF) return set_error(UNO_ERR_UNSUPPORTED, "too many rows");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)S;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(N * S));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, static_cast<const T*>(logits), p),
                      "launch(token logprobs)");
}

template <typename T>
uno_status grad_launch(const void* logits, void* grad, int64_t N, GradArgs p, cudaStream_t stream) {
    const int64_t pieces = p.V / kVec<T> + 1, per = kGradThreads * kGradPieces;
    const int64_t chunks = (pieces + per - 1) / per;
    if (chunks * N > 0x7FFFFFFF) return set_error(UNO_ERR_UNSUPPORTED, "too many logits for one launch");
    p.chunks = (int)chunks;
    logprobs_grad_kernel<T><<<(unsigned)(chunks * N), kGradThreads, 0, stream>>>(static_cast<const T*>(logits),
                                                                                static_cast<T*>(grad), p);
    return check_cuda(cudaGetLastError(), "launch(token logprobs gradient)");
}

uno_status check_rows(uno_dtype dtype, int64_t N, int64_t V, float temperature) {
    if (bad_dtype(dtype)) return set_error(UNO_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (N < 0 || V < 1) return set_error(UNO_ERR_INVALID_ARG, "need N >= 0 and V >= 1");
    if (!(temperature > 0.f) || !(temperature < INFINITY))
        return set_error(UNO_ERR_INVALID_ARG, "temperature must be positive and finite");
    if (temperature < 1e-30f) return set_error(UNO_ERR_UNSUPPORTED, "temperature >= 1e-30 is supported");
    if (V > 0x7FFFF000) return set_error(UNO_ERR_UNSUPPORTED, "V < 2^31 - 4096 is supported");
    if (N > 0x7FFFFFFF || (double)N * (double)V >= 1099511627776.0)
        return set_error(UNO_ERR_UNSUPPORTED, "N < 2^31 and N * V < 2^40 are supported");
    return UNO_OK;
}

}  // namespace
}  // namespace uno

extern "C" uno_status uno_token_logprobs(const void* logits, uno_dtype dtype, int64_t N, int64_t V, float temperature,
                                         const int32_t* tokens, int32_t top_n, float* out_logprob, float* out_entropy,
                                         float* out_stats, int32_t* out_top_ids, float* out_top_logprobs,
                                         uno_stream_t stream) {
    using namespace uno;
    uno_status s = check_rows(dtype, N, V, temperature);
    if (s != UNO_OK) return s;
    if (top_n < 0) return set_error(UNO_ERR_INVALID_ARG, "top_n must be >= 0");
    if (top_n > kMaxTop) return set_error(UNO_ERR_UNSUPPORTED, "top_n <= %d is supported", kMaxTop);
    if (N == 0) return UNO_OK;
    if (!logits) return set_error(UNO_ERR_INVALID_ARG, "logits is NULL");
    if (out_logprob && !tokens) return set_error(UNO_ERR_INVALID_ARG, "out_logprob needs tokens");
    if ((top_n > 0) != (out_top_ids != nullptr) || (top_n > 0) != (out_top_logprobs != nullptr))
        return set_error(UNO_ERR_INVALID_ARG, "out_top_ids and out_top_logprobs are given exactly when top_n > 0");
    if (!out_logprob && !out_entropy && !out_stats && !out_top_ids)
        return set_error(UNO_ERR_INVALID_ARG, "at least one output is required");
    const void* ptrs[] = {logits, tokens, out_logprob, out_entropy, out_stats, out_top_ids, out_top_logprobs};
    for (const void* p : ptrs)
        if (off16(p)) return set_error(UNO_ERR_UNSUPPORTED, "tensor pointers must be 16-byte aligned");
    const float c = (float)(1.4426950408889634 / (double)temperature);
    const Args a{V, c, (float)(4 * 1.4426950408889634 / (double)temperature), 4.0f / temperature,
                 c > kMinC && c < kMaxC, tokens, top_n, out_logprob, out_entropy, out_stats, out_top_ids,
                 out_top_logprobs};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == UNO_F32 ? logprobs_launch<float>(logits, N, a, st)
                            : logprobs_launch<__nv_bfloat16>(logits, N, a, st);
}

extern "C" uno_status uno_token_logprobs_grad(const void* logits, uno_dtype dtype, int64_t N, int64_t V,
                                              float temperature, const int32_t* tokens, const float* stats,
                                              const float* entropy, const float* grad_logprob,
                                              const float* grad_entropy, void* grad_logits, uno_stream_t stream) {
    using namespace uno;
    uno_status s = check_rows(dtype, N, V, temperature);
    if (s != UNO_OK) return s;
    if (N == 0) return UNO_OK;
    if (!logits || !stats || !grad_logits)
        return set_error(UNO_ERR_INVALID_ARG, "logits, stats and grad_logits are required");
    if (!grad_logprob && !grad_entropy)
        return set_error(UNO_ERR_INVALID_ARG, "grad_logprob or grad_entropy is required");
    if (grad_logprob && !tokens) return set_error(UNO_ERR_INVALID_ARG, "grad_logprob needs tokens");
    if (grad_entropy && !entropy) return set_error(UNO_ERR_INVALID_ARG, "grad_entropy needs entropy");
    const void* ptrs[] = {logits, tokens, stats, entropy, grad_logprob, grad_entropy, grad_logits};
    for (const void* p : ptrs)
        if (off16(p)) return set_error(UNO_ERR_UNSUPPORTED, "tensor pointers must be 16-byte aligned");
    const GradArgs a{V, (float)(4 * 1.4426950408889634 / (double)temperature), 4.0f / temperature, tokens, stats,
                     entropy, grad_logprob, grad_entropy, 0};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == UNO_F32 ? grad_launch<float>(logits, grad_logits, N, a, st)
                            : grad_launch<__nv_bfloat16>(logits, grad_logits, N, a, st);
}
