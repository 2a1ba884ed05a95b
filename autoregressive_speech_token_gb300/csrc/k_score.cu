// sd_score_rows: log probability and rank of a given token, entropy, and the most
// probable alternatives of rows of logits.
//
// With d_j = z_j - m, m the row's largest logit, S = sum e^(d/T) and D = sum d e^(d/T),
//   log p_j = d_j / T - log S,   H = log S - D / (S T)   (both terms of H are >= 0: nothing cancels).
//
// A row is read from memory once, in 16-byte vectors that cp.async brings into a ring in shared memory, eight of a thread
// in flight.  The first four of every thread are spread over the whole part: their largest entry is what the block's sums are
// relative to (d_j is formed first: exact where it counts; a thread that meets a larger entry shrinks what it has).
// Long rows, where rows are fewer than the SMs, are cut over a thread-block cluster, whose blocks exchange their maxima,
// sums and best entries through distributed shared memory.
//
// The first n entries of (z descending, index ascending): every entry is the 64-bit key (order of z, ~index), 0 if it is
// no alternative.  The best keys of groups of four threads in the first round are ranked among each other.  The n-th of
// them is a bound: at least n keys reach it.  Vectors that reach it, a few n, are put aside as the row passes; their keys
// are ranked at the end, each against all.  Where too much reaches it (a rising row, a mask over most of the first
// round), the bound is taken of the whole part and what reaches it is read again; where that is still too much, the n best
// are taken one after the other.
//
// Most vectors are below the watched bound (the smallest of the maximum, the n-th best and the token's logit) and
// cost only their sums, with two fp32 operations an instruction where pairs allow.
//
// Measured (token, rank, entropy and best entries of every row): 16 rows of 2048 6 us, a chain of exchanges; 800 of 8194
// fp32 with 20 wanted 19 us = 1.4 TB/s, where the ranking and the chain of a short row bound it (13.3 without token and
// best); 1021 of 131075 bf16 with 8 wanted 83 us = 3.2 TB/s, where the issue of instructions does (78 % busy, 144 for a warp's
// 32 vectors, 90 of them for the sums; the bound of exp2 is 28 us); fp32 without token and best 101 us = 5.3 TB/s.
#include <algorithm>

#include "pages_dev.cuh"
namespace sd {
namespace {

// Where an access refused itself: the address, for a debugger.  Every address below is aligned by construction (the same
// code on the host, under a sanitizer, shows no other), yet without these checks one block of one row with token -1
// ended with a "misaligned address" on GB300 (CUDA 13.0), and with them nothing is ever refused.  They stay until the
// cause is known.
__device__ unsigned long long g_refused[32];
__device__ __forceinline__ bool aligned(const void* p, int n, int access) {
    if ((reinterpret_cast<unsigned long long>(p) & (n - 1)) == 0) return true;
    g_refused[access] = reinterpret_cast<unsigned long long>(p);
    return false;
}

constexpr int kMaxTop = 32, kMaxCluster = 16, kList = 512;
constexpr int kMaxVocab = 262144;

struct ScoreArgs {
    const void* z;
    const int32_t* token;
    float *logp, *entropy, *top_logp;
    int32_t *rank, *top_id;
    int64_t stride;
    int32_t V, top;
    float T, c;                                            // temperature; log2(e) / T
};

__device__ __forceinline__ float ex2_(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan_(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// Order of the values as unsigned numbers (both zeros alike); 0: no alternative (-inf, NaN)
__device__ __forceinline__ uint32_t order_of(float x) {
    if (!(x > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o); }

// two fp32 operations an instruction
__device__ __forceinline__ float2 add2_(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2_(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2_(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}

using Key = unsigned long long;
__device__ __forceinline__ Key key_of(float x, int32_t index) {
    const uint32_t o = order_of(x);
    return o ? (Key)o << 32 | (uint32_t)~index : 0;
}
__device__ __forceinline__ Key max_key(Key a, Key b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t remote(uint32_t addr, int rank) {
    uint32_t x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(addr), "r"(rank));
    return x;
}
__device__ __forceinline__ Key remote_key(uint32_t addr) {
    Key x;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ float remote_float(uint32_t addr) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_size() {
    uint32_t x;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(x));
    return (int)x;
}
__device__ __forceinline__ int cluster_rank() {
    uint32_t x;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(x));
    return (int)x;
}

template <typename T>
struct Type {
    static constexpr int kN = 16 / sizeof(T);              // elements of a 16-byte vector
    static constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    static constexpr uint32_t kLow = sizeof(T) == 4 ? 0xff800000u : kBf ? 0xff80ff80u : 0xfc00fc00u;   // -inf
    using Pair = std::conditional_t<kBf, __nv_bfloat162, __half2>;
};
__device__ __forceinline__ uint32_t word_of(const uint4& w, int e) { return e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w; }
// Element e of a vector
template <typename T>
__device__ __forceinline__ float element(const uint4& w, int e) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(word_of(w, e));
    else {
        const uint32_t x = word_of(w, e >> 1);
        if constexpr (Type<T>::kBf) return __uint_as_float((e & 1) ? x & 0xffff0000u : x << 16);
        else return __half2float(__ushort_as_half((unsigned short)((e & 1) ? x >> 16 : x)));
    }
}
// The larger of each two, of a number and NaN the number
template <typename T>
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    else {
        using Pair = typename Type<T>::Pair;
        const Pair m = __hmax2(*reinterpret_cast<const Pair*>(&a), *reinterpret_cast<const Pair*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
}

// The number of the type before x (x above -inf)
template <typename T>
__device__ __forceinline__ float before_of(float x) {
    constexpr uint32_t kStep = sizeof(T) == 4 ? 1u : Type<T>::kBf ? 0x10000u : 0;
    if constexpr (kStep != 0) {
        const uint32_t b = __float_as_uint(x);
        if (x == 0.f) return __uint_as_float(0x80000000u | kStep);
        return __uint_as_float((b >> 31) ? b + kStep : b - kStep);
    } else {
        const unsigned short b = __half_as_ushort(__float2half_rn(x));
        if (x == 0.f) return __half2float(__ushort_as_half(0x8001));
        return __half2float(__ushort_as_half((unsigned short)((b >> 15) ? b + 1 : b - 1)));
    }
}
// A number of the type twice
template <typename T>
__device__ __forceinline__ typename Type<T>::Pair pair_of(float x) {
    if constexpr (Type<T>::kBf) return __float2bfloat162_rn(x);
    else return __float2half2_rn(x);
}
__device__ __forceinline__ float number(float x) { return x; }
__device__ __forceinline__ float number(__half x) { return __half2float(x); }
__device__ __forceinline__ float number(__nv_bfloat16 x) { return __bfloat162float(x); }

// The elements of a vector that the row has, the others -inf
template <typename T>
__device__ __forceinline__ uint4 load_edge(const T* row, int first, int32_t V) {
    uint32_t w[4] = {Type<T>::kLow, Type<T>::kLow, Type<T>::kLow, Type<T>::kLow};
#pragma unroll
    for (int e = 0; e < Type<T>::kN; ++e) {
        const int j = first + e;
        if (j < 0 || j >= V) continue;
        if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(row[j]);
        else {
            const uint32_t b = *reinterpret_cast<const unsigned short*>(row + j);
            w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | b << 16 : (w[e >> 1] & 0xffff0000u) | b;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kStages = 8;                                 // vectors of a thread in flight, in shared memory
constexpr int kPutAside = 128;                            // vectors that may reach the first bound before it is raised
constexpr int kFirst = 4;                                  // of which the bound is taken

template <typename T, int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) k_score(const ScoreArgs a) {
    constexpr int kN = Type<T>::kN, kWarps = kThreads / 32, kGroups = kThreads / 4, kHits = 2 * kThreads;
    __shared__ uint4 s_hit[kHits];                         // vectors with an entry that reaches the bound
    __shared__ int s_hit_j[kHits];                         // and their first entry
    __shared__ Key s_best[2 * kGroups], s_top[kMaxTop], s_tau;
    __shared__ float s_max[kWarps], s_S[kWarps], s_D[kWarps], s_mine[3];           // s_mine: this block's maximum, S, D
    __shared__ int s_ahead[kWarps], s_mine_ahead, s_count, s_keys;
    extern __shared__ uint4 s_ring[];                      // [kStages][kThreads]: a thread reads back only what it copied
    Key* s_list = reinterpret_cast<Key*>(s_ring);          // keys in its place, once the row has passed
    static_assert(kStages * 2 * kThreads >= kList, "");
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = kCluster ? cluster_size() : 1, c = kCluster ? cluster_rank() : 0;
    const int64_t row = blockIdx.x / C;
    const T* z = static_cast<const T*>(a.z) + row * a.stride;
    const int lead = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));     // elements between a 16-byte boundary and the row

    // ---- this block's vectors v0, v0 + 1, ..., nv of them; vector v begins with element v kN - lead.  A thread takes vector
    // tid of every kThreads; the first kFirst of its turns are from all over the part.  The row's ragged ends are an extra
    // vector of two threads.
    const int all = (a.V + lead + kN - 1) / kN, each = (all + C - 1) / C, v0 = c * each, nv = min(each, all - v0);
    const int inner = lead > 0, whole = (a.V + lead) / kN; // vectors [inner, whole) lie within the row
    const int turns = max((nv + kThreads - 1) / kThreads, 0), quarter = (turns + kFirst - 1) / kFirst;
    const int low = max(v0, inner), count_v = max(min(whole, v0 + nv) - low, 0);
    // vector of turn x (< kFirst) of round q, and whether it is a whole one of this part
    auto vector_of = [&](int q, int x) { return v0 + (x * quarter + q) * kThreads + tid; };
    auto there = [&](int v) { return (uint32_t)(v - low) < (uint32_t)count_v; };
    auto index_of = [&](int v) { return v * kN - lead; };  // of a vector's first element
    static_assert(kStages == 2 * kFirst, "two rounds in flight");
    auto slot = [&](int q, int x) { return s_ring + ((q & 1) * kFirst + x) * kThreads + tid; };
    // a round's vectors; places without one hold -inf
    const bool sound = count_v == 0 || aligned(z + index_of(low), 16, 0);
    auto copy = [&](int q) {
        if (q < quarter) {
#pragma unroll
            for (int x = 0; x < kFirst; ++x) {
                const int v = vector_of(q, x);
                if (there(v) && sound)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(slot(q, x))), "l"(z + index_of(v)) : "memory");
                else
                    *slot(q, x) = make_uint4(Type<T>::kLow, Type<T>::kLow, Type<T>::kLow, Type<T>::kLow);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy(0);
    copy(1);
    uint4 edge = make_uint4(Type<T>::kLow, Type<T>::kLow, Type<T>::kLow, Type<T>::kLow);
    int edge_j = 0;
    bool has_edge = false;
    {
        const int v = tid == 0 && inner ? 0 : tid == 1 && whole * kN < a.V + lead ? whole : -1;
        // a row within one vector: its end is its beginning
        if (v >= v0 && v < v0 + nv && !(v == whole && tid == 1 && whole == 0 && inner)) {
            edge_j = index_of(v);
            edge = load_edge(z, edge_j, a.V);
            has_edge = true;
        }
    }
    const int32_t token = a.token && aligned(a.token + row, 4, 1) ? a.token[row] : -1;
    const bool given = (uint32_t)token < (uint32_t)a.V;
    const float zt = given && aligned(z + token, sizeof(T), 2) ? number(z[token]) : -INFINITY;

    // ---- running maximum and sums, and how many entries are ahead of the token.  The difference to the maximum is formed
    // first: exact where it counts, whatever the logits' size.  Nothing 200 / c below it counts, which keeps it finite.
    const float least = -200.f / a.c;
    float m = -INFINITY, S = 0.f, D = 0.f;                 // m: what the sums are relative to
    int ahead = 0;
    auto largest = [&](const uint4& w) {
        const uint32_t mw = max_words<T>(max_words<T>(w.x, w.y), max_words<T>(w.z, w.w));
        return sizeof(T) == 4 ? __uint_as_float(mw) : fmaxf(element<T>(make_uint4(mw, 0, 0, 0), 0), element<T>(make_uint4(mw, 0, 0, 0), 1));
    };
    // the sums of a vector whose largest entry m has seen: two fp32 operations an instruction
    float2 S2 = make_float2(0.f, 0.f), D2 = S2;
    auto add = [&](const uint4& w, float2 ref) {
        const float2 c2 = make_float2(a.c, a.c);
#pragma unroll
        for (int e = 0; e < kN; e += 2) {
            float2 d = add2_(make_float2(element<T>(w, e), element<T>(w, e + 1)), ref);
            d.x = max_nan_(d.x, least);
            d.y = max_nan_(d.y, least);
            float2 p = mul2_(d, c2);
            p.x = ex2_(p.x);
            p.y = ex2_(p.y);
            S2 = add2_(S2, p);
            D2 = fma2_(d, p, D2);
        }
    };
    // entries of a vector, the first of them entry j, that are ahead of the token.  16-bit ones two at a time: 1 or 0 each,
    // added up in their own type (at most 4 a vector and half, 33 vectors before they are taken out: bf16 holds whole numbers up to 256)
    using Pair = typename Type<T>::Pair;
    Pair ahead2 = {};
    // x >= zt is x > (what comes before zt in the type): entries before the token and behind it differ in one number
    const float before_zt = before_of<T>(zt);
    const Pair zt2 = pair_of<T>(zt), before_zt2 = pair_of<T>(before_zt);
    const int before_end = zt > -INFINITY ? token : -kN;   // (what lies before the row is -inf: not ahead of a finite logit)
    auto count = [&](const uint4& w, int j) {
        const bool behind = j > token, before = j + kN <= before_end;
        if (behind || before) {
            if constexpr (sizeof(T) == 4) {
                const float x = behind ? zt : before_zt;
#pragma unroll
                for (int e = 0; e < kN; ++e) ahead += element<T>(w, e) > x;
            } else {
                const Pair x = behind ? zt2 : before_zt2;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t u = word_of(w, e);
                    ahead2 = __hadd2(ahead2, __hgt2(*reinterpret_cast<const Pair*>(&u), x));
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const float x = element<T>(w, e);
                ahead += x > zt || (x == zt && (uint32_t)(j + e) < (uint32_t)token);
            }
        }
    };
    auto flush = [&]() {
        if constexpr (sizeof(T) == 2) {
            ahead += (int)(__low2float(ahead2) + __high2float(ahead2));
            ahead2 = Pair{};
        }
    };
    // A vector with an entry that reaches the bound's value is put aside: few are, and a warp waits for each of its lanes
    auto collect = [&](const uint4& w, int j) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kHits && aligned(s_hit + at, 16, 6)) {
            s_hit[at] = w;
            s_hit_j[at] = j;
        }
    };
    // The keys of what was put aside that reach the bound tau; more than kList if there are too many
    auto keys_of_hits = [&](Key tau) -> int {
        const int n = s_count;
        if (n > kHits) return kList + 1;
        for (int i = tid; i < n * kN; i += kThreads) {
            const T x = reinterpret_cast<const T*>(s_hit)[i];
            const Key k = key_of(number(x), s_hit_j[i / kN] + i % kN);
            if (k < tau) continue;
            const int at = atomicAdd(&s_keys, 1);
            if (at < kList && aligned(s_list + at, 8, 13)) s_list[at] = k;
        }
        __syncthreads();
        return s_keys;
    };
    // The n-th of the groups' best keys so far, 1 if there are fewer: at least n entries reach it, or all do
    auto bound_of = [&](const uint4& best, int best_j, float m) -> Key {
        int at = 0;
#pragma unroll
        for (int e = kN - 1; e >= 0; --e) at = element<T>(best, e) == m ? best_j + e : at;
        Key mine = key_of(m, at);
        mine = max_key(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
        mine = max_key(mine, __shfl_xor_sync(0xffffffffu, mine, 2));
        if ((tid & 3) == 0 && aligned(s_best + (tid >> 2), 8, 4)) s_best[tid >> 2] = mine;
        if (tid == 0) {
            s_count = s_keys = 0;
            s_tau = 0;
        }
        if (tid < kMaxTop && aligned(s_top + tid, 8, 5)) s_top[tid] = 0;
        __syncthreads();
        // group tid / 4 against a quarter of the groups
        const Key key = s_best[tid >> 2];
        int before = 0;
#pragma unroll 8
        for (int g = 0; g < kGroups / 4; ++g) before += s_best[g * 4 + (tid & 3)] > key;
        before += __shfl_xor_sync(0xffffffffu, before, 1);
        before += __shfl_xor_sync(0xffffffffu, before, 2);
        if ((tid & 3) == 0 && key && before == a.top - 1) s_tau = key;          // keys are distinct
        __syncthreads();
        return max_key(s_tau, 1);
    };
    // A higher bound while a long part passes: the n-th of the best keys of the vectors put aside so far
    auto higher_bound = [&](Key tau) -> Key {
        __syncthreads();
        const int n = s_count;
        if (n > 2 * kGroups) return tau;
        if (tid < n && aligned(s_best + tid, 8, 14)) {
            Key most = 0;
#pragma unroll
            for (int e = 0; e < kN; ++e) most = max_key(most, key_of(element<T>(s_hit[tid], e), s_hit_j[tid] + e));
            s_best[tid] = most;
        }
        __syncthreads();
        for (int i0 = 0; i0 < n; i0 += kGroups) {
            const int i = i0 + (tid >> 2);
            const Key key = s_best[min(i, n - 1)];
            int before = 0;
#pragma unroll 4
            for (int j = tid & 3; j < n; j += 4) before += s_best[j] > key;
            before += __shfl_xor_sync(0xffffffffu, before, 1);
            before += __shfl_xor_sync(0xffffffffu, before, 2);
            if ((tid & 3) == 0 && i < n && key && before == a.top - 1) s_tau = key;
        }
        __syncthreads();
        return max_key(s_tau, tau);
    };
    auto value_bound = [&](Key tau) { return tau > 1 ? value_of((uint32_t)(tau >> 32)) : -INFINITY; };

    // The sums are relative to the block's largest entry among the first turns.  Where a larger one comes, what was summed
    // shrinks.
    auto raise = [&](float top) {
        const float by = fmaxf(m - top, least), f = ex2_(by * a.c);
        D = (D + D2.x + D2.y + (S + S2.x + S2.y) * by) * f;
        S = (S + S2.x + S2.y) * f;
        S2 = D2 = make_float2(0.f, 0.f);
        m = top;
    };
    auto ring = [&](int q, int x) { return *slot(q, x); };
    Key tau = 0;
    float bound = INFINITY;                                // nothing is collected without `top`
    {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        uint4 best = edge;
        int best_j = edge_j;
        float top = largest(edge);
#pragma unroll 1
        for (int x = 0; x < kFirst && quarter; ++x) {
            const uint4 w = ring(0, x);
            const float y = largest(w);
            if (y > top || !(top > -INFINITY)) {
                best = w;
                best_j = index_of(vector_of(0, x));
                top = y;
            }
        }
        if (!(top > -INFINITY)) top = -INFINITY;
        m = top;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0 && aligned(s_max + warp, 4, 3)) s_max[warp] = m;
        if (a.top) tau = bound_of(best, best_j, top);
        else __syncthreads();
        if (a.top) bound = value_bound(tau);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_max[w]);
        __syncthreads();                                   // s_max is used again
    }
    // A token below the best entries has some ahead of it in most vectors: counted in all of them without a look (1021 rows of
    // 131075 bf16 87 -> 83 us)
    const bool often = given && zt < fminf(m, bound);
    const float rare = given && !often ? zt : INFINITY;
    float watch = fminf(fminf(m, bound), rare), ref = m == -INFINITY ? 0.f : -m;
    auto visit = [&](const uint4& w, int j) {
        const float top = largest(w);
        if (often) count(w, j);
        if (top >= watch) {                                // most vectors have nothing to be looked at
            if (top > m) {
                raise(top);
                ref = -m;
            }
            if (top >= rare) count(w, j);
            if (top >= bound) collect(w, j);
            watch = fminf(fminf(m, bound), rare);
        }
        add(w, make_float2(ref, ref));
    };
    if (has_edge) visit(edge, edge_j);
#pragma unroll 1
    for (int q = 0; q < quarter; ++q) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll 1
        for (int x = 0; x < kFirst; ++x) {
            const int v = vector_of(q, x);
            if (there(v)) visit(ring(q, x), index_of(v));
        }
        copy(q + 2);
        if ((q & 7) == 7) flush();
        // About top_n times the number of rounds will have reached the first round's bound.  Behind rounds 4 and 16 it is
        // raised, which stalls the block for 1.5 us: 1021 rows of 131075 fp32 with 20 wanted 190 -> 142 us, but of bf16 (half
        // the rounds) with 8 wanted 85 -> 90
        if (a.top * quarter > kPutAside && (q == 3 || q == 15) && 2 * (q + 1) <= quarter) {
            tau = higher_bound(tau);
            bound = value_bound(tau);
            watch = fminf(fminf(m, bound), rare);
        }
    }
    flush();
    S += S2.x + S2.y;
    D += D2.x + D2.y;

    // ---- the block's maximum, and its sums
    float mb = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    if (lane == 0 && aligned(s_max + warp, 4, 3)) s_max[warp] = mb;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mb = fmaxf(mb, s_max[w]);
    if (m != mb) {                                         // (a thread without a number may have seen NaN: kept)
        const float by = m == -INFINITY ? 0.f : fmaxf(m - mb, least), f = ex2_(by * a.c);
        D = (D + S * by) * f;
        S *= f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, o);
        D += __shfl_xor_sync(0xffffffffu, D, o);
    }
    ahead = __reduce_add_sync(0xffffffffu, ahead);
    if (lane == 0) {
        s_S[warp] = S;
        s_D[warp] = D;
        s_ahead[warp] = ahead;
    }

    // ---- the block's first entries
    if (a.top) {
        int n = keys_of_hits(tau);
        if (n > kList) {
            // the first batch's bound let too many through (few entries there, or a rising row): the whole part's bound
            __syncthreads();
            uint4 best = edge;
            int best_j = edge_j;
            float top = largest(edge);
#pragma unroll 1
            for (int v = v0 + tid; v < v0 + nv; v += kThreads) {
                if (!there(v)) continue;
                const uint4 x = *reinterpret_cast<const uint4*>(z + index_of(v));
                const float y = largest(x);
                if (y > top || !(top > -INFINITY)) {
                    best = x;
                    best_j = index_of(v);
                    top = y;
                }
            }
            if (!(top > -INFINITY)) top = -INFINITY;
            tau = bound_of(best, best_j, top);
            bound = value_bound(tau);
            if (top >= bound) {
                if (largest(edge) >= bound) collect(edge, edge_j);
#pragma unroll 1
                for (int v = v0 + tid; v < v0 + nv; v += kThreads) {
                    if (!there(v)) continue;
                    const uint4 x = *reinterpret_cast<const uint4*>(z + index_of(v));
                    if (largest(x) >= bound) collect(x, index_of(v));
                }
            }
            __syncthreads();
            n = keys_of_hits(tau);
        }
        if (n <= kList) {
            // four threads to a key, a quarter of the others each
            for (int i0 = 0; i0 < n; i0 += kThreads / 4) {
                const int i = i0 + (tid >> 2);
                const Key x = s_list[min(i, n - 1)];
                int r = 0;
#pragma unroll 4
                for (int j = tid & 3; j < n; j += 4) r += s_list[j] > x;
                r += __shfl_xor_sync(0xffffffffu, r, 1);
                r += __shfl_xor_sync(0xffffffffu, r, 2);
                if ((tid & 3) == 0 && i < n && r < a.top && aligned(s_top + r, 8, 7)) s_top[r] = x;
            }
        } else {
            Key last = ~(Key)0;
            for (int k = 0; k < a.top; ++k) {
                Key most = 0;
#pragma unroll 1
                for (int v = v0 + tid - kThreads; v < v0 + nv; v += kThreads) {
                    const bool first = v < v0 + tid;       // the extra vector
                    if (!first && !there(v)) continue;
                    const uint4 w = first ? edge : *reinterpret_cast<const uint4*>(z + index_of(v));
#pragma unroll
                    for (int e = 0; e < kN; ++e) {
                        const Key x = key_of(element<T>(w, e), (first ? edge_j : index_of(v)) + e);
                        if (x < last) most = max_key(most, x);
                    }
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) most = max_key(most, __shfl_xor_sync(0xffffffffu, most, o));
                __syncthreads();
                if (lane == 0) s_list[warp] = most;
                __syncthreads();
                for (int w = 0; w < kWarps; ++w) most = max_key(most, s_list[w]);
                if (tid == 0) s_top[k] = most;
                last = most;
                if (!most) break;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        float s = 0.f, d = 0.f;
        int n = 0;
        for (int w = 0; w < kWarps; ++w) {
            s += s_S[w];
            d += s_D[w];
            n += s_ahead[w];
        }
        s_mine[0] = mb;
        s_mine[1] = s;
        s_mine[2] = d;
        s_mine_ahead = n;
    }

    // ---- the row's: the cluster's first block gathers
    Key* s_all = s_list;                                  // [block][kMaxTop]
    static_assert(kList >= kMaxCluster * kMaxTop, "the lists of all blocks");
    float m_of = -INFINITY, s_of = 0.f, d_of = 0.f;        // of block `lane`
    int ahead_of = 0;
    if constexpr (kCluster) {
        cluster_sync();
        if (c == 0) {
            for (int i = tid; i < C * a.top; i += kThreads) {
                const int r = i / a.top, k = i - r * a.top;
                s_all[r * kMaxTop + k] = remote_key(remote(smem_addr(s_top + k), r));
            }
            if (lane < C) {
                m_of = remote_float(remote(smem_addr(s_mine), lane));
                s_of = remote_float(remote(smem_addr(s_mine + 1), lane));
                d_of = remote_float(remote(smem_addr(s_mine + 2), lane));
                ahead_of = __float_as_int(remote_float(remote(smem_addr(&s_mine_ahead), lane)));
            }
        }
        cluster_sync();                                    // nothing of another block is read behind this
    } else {
        __syncthreads();
        if (lane == 0) {
            m_of = s_mine[0];
            s_of = s_mine[1];
            d_of = s_mine[2];
            ahead_of = s_mine_ahead;
        }
    }
    if (c != 0) return;
    float M = m_of;
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    {
        const float by = m_of == -INFINITY ? 0.f : max_nan_(m_of - M, least), f = ex2_(by * a.c);
        S = s_of * f;
        D = (d_of + s_of * by) * f;
        ahead = ahead_of;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, o);
        D += __shfl_xor_sync(0xffffffffu, D, o);
    }
    ahead = __reduce_add_sync(0xffffffffu, ahead);
    const float log_s = logf(S);
    // log p of a logit; a row without a finite logit has none
    auto log_p = [&](float x) { return S == 0.f ? -INFINITY : (x - M) / a.T - log_s; };
    if (tid == 0) {
        if (a.logp && aligned(a.logp + row, 4, 8)) a.logp[row] = given ? log_p(zt) : 0.f;
        if (a.rank && aligned(a.rank + row, 4, 9)) a.rank[row] = given ? ahead : -1;
        if (a.entropy && aligned(a.entropy + row, 4, 10)) a.entropy[row] = S == 0.f ? 0.f : log_s - D / S / a.T;
    }
    if (!a.top) return;
    auto put = [&](int r, Key x) {
        const int64_t at = row * a.top + r;
        if (!aligned(a.top_id + at, 4, 11) || !aligned(a.top_logp + at, 4, 12)) return;
        a.top_id[at] = x ? (int32_t)~(uint32_t)x : -1;
        a.top_logp[at] = x ? log_p(value_of((uint32_t)(x >> 32))) : -INFINITY;
    };
    if constexpr (!kCluster) {
        if (tid < a.top) put(tid, s_top[tid]);
    } else {
        // keys of all blocks: the place in the own list, and how many of each other list are ahead
        for (int i = tid; i < C * a.top; i += kThreads) {
            const int r = i / a.top, k = i - r * a.top;
            const Key x = s_all[r * kMaxTop + k];
            if (!x) continue;
            int place = k;
            for (int q = 0; q < C && place < a.top; ++q) {
                if (q == r) continue;
                int lo = 0, hi = a.top;                        // sorted, falling
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (s_all[q * kMaxTop + mid] > x) lo = mid + 1;
                    else hi = mid;
                }
                place += lo;
            }
            if (place < a.top) put(place, x);
        }
        // places that no entry takes
        int have = 0;
        for (int q = 0; q < C; ++q) {
            int lo = 0, hi = a.top;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s_all[q * kMaxTop + mid]) lo = mid + 1;
                else hi = mid;
            }
            have += lo;
        }
        if (tid < a.top && tid >= have) put(tid, 0);
    }
}

template <typename T, int kThreads, bool kCluster>
cudaError_t launch_row(const ScoreArgs& a, int rows, int C, cudaStream_t st) {
    auto kernel = k_score<T, kThreads, kCluster>;
    constexpr int kSmem = kStages * kThreads * 16;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (!kCluster) return launch_k(kernel, dim3((unsigned)rows), dim3(kThreads), kSmem, st, a);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)rows * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = use_pdl() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <typename T, int kThreads>
cudaError_t launch(const ScoreArgs& a, int rows, int C, cudaStream_t st) {
    return C > 1 ? launch_row<T, kThreads, true>(a, rows, C, st) : launch_row<T, kThreads, false>(a, rows, C, st);
}

template <typename T>
cudaError_t choose(const ScoreArgs& a, int rows, int sms, cudaStream_t st) {
    const int64_t bytes = ((int64_t)a.V + 2 * Type<T>::kN - 2) / Type<T>::kN * 16;      // a row may begin and end inside a vector
    // Few rows: over more SMs, as long as a block keeps 16 KB.  The part of a block is streamed, whatever its length.
    int C = 1;
    while (C < kMaxCluster && (int64_t)rows * C * 2 <= 2 * sms && bytes > (int64_t)C * 16384) C *= 2;
    if ((int64_t)rows * C > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t part = bytes / C, blocks = (int64_t)rows * C;
    // 128, 256 or 512 threads to a block.  Smaller ones finish more rows side by side, and have fewer bounds to rank: 1000 rows
    // of 2050 fp32 13.3 us by 256, 11.6 by 128; 1000 of 16386 40.4 by 512, 32.8 by 256.  Few rows want larger ones (320 of
    // 8194: 17.5 us by 128, 11.5 by 256), and so do long parts, where the first round shows less of the row (700 of 32000 with
    // 20 wanted: 39.5 by 512, 40 to 47 by 256).
    if (part <= 16384 && blocks > 4 * sms) return launch<T, 128>(a, rows, C, st);
    return part <= 98304 && blocks > 2 * sms ? launch<T, 256>(a, rows, C, st) : launch<T, 512>(a, rows, C, st);
}

}  // namespace
}  // namespace sd

extern "C" int sd_score_rows(const void* logits_dev, int64_t stride, int32_t dtype, int32_t rows, int32_t V,
                             float temperature, const int32_t* token_dev, float* logp_dev, int32_t* rank_dev,
                             float* entropy_dev, int32_t top_n, int32_t* top_id_dev, float* top_logp_dev, void* stream) {
    using namespace sd;
    static const char* who = "sd_score_rows";
    if (rows == 0) return SD_OK;
    const int b = dtype == SD_E4M3 ? 0 : dtype_bytes(dtype);
    if (!b) return op_fail(SD_ERR_INVALID_ARG, "%s: type %d is not SD_F32, SD_F16 or SD_BF16", who, dtype);
    if (rows < 0 || V < 1 || top_n < 0) return op_fail(SD_ERR_INVALID_ARG, "%s: rows %d, V %d, top_n %d", who, rows, V, top_n);
    if (V > kMaxVocab || top_n > kMaxTop)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: V %d (up to %d), top_n %d (up to %d)", who, V, kMaxVocab, top_n, kMaxTop);
    if (!logits_dev || (reinterpret_cast<uintptr_t>(logits_dev) % b))
        return op_fail(SD_ERR_INVALID_ARG, "%s: logits_dev is NULL or not aligned to its elements", who);
    if (rows > 1 && stride < V) return op_fail(SD_ERR_INVALID_ARG, "%s: stride %lld is below V %d", who, (long long)stride, V);
    if (!(temperature >= 1e-30f && temperature <= 1e30f))
        return op_fail(SD_ERR_INVALID_ARG, "%s: temperature %g", who, (double)temperature);
    if (!token_dev && (logp_dev || rank_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: logp_dev and rank_dev need token_dev", who);
    if (top_n > 0 && (!top_id_dev || !top_logp_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: top_id_dev or top_logp_dev is NULL", who);
    ScoreArgs a = {};
    a.z = logits_dev; a.token = token_dev; a.logp = logp_dev; a.entropy = entropy_dev; a.top_logp = top_logp_dev;
    a.rank = rank_dev; a.top_id = top_id_dev; a.stride = rows > 1 ? stride : 0; a.V = V; a.top = top_n; a.T = temperature;
    a.c = (float)(1.4426950408889634 / (double)temperature);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (e == cudaSuccess)
        e = dtype == SD_F32 ? choose<float>(a, rows, sms, st)
            : dtype == SD_F16 ? choose<__half>(a, rows, sms, st) : choose<__nv_bfloat16>(a, rows, sms, st);
    if (e != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return SD_OK;
}

