// distill.cu -- bakron_distill: the distillation loss from a teacher's top logits and its gradient.
//
//   q = softmax(z / tau),  p_j = exp(t_j / tau - T),
//   loss = w sum_j p_j (log p_j - log q_{i_j}),   dz_i = (w / tau) (M q_i - sum_{j: i_j = i} p_j)
//
// Bound by bytes: a row of the vocabulary read once, and written once with the gradient. What stands
// against it is the chain of a row: its list (index, then the logit there), its statistics, a
// barrier, and only then its gradient; about 5 us, in which an SM could move 200 KB. So:
//
//   * Many rows (distill_rows_kernel): blocks stay on the GPU and go from row to row. A thread keeps
//     its first vectors of a row in shared memory, brought there by cp.async during the row before (as
//     soon as that row's own are written out); what does not fit is streamed, and read again from
//     L2 for the gradient. One warp goes through the teacher's lists a row ahead. The barriers are
//     named ones: between the data warps, and between them and the list's warp.
//   * Few rows (distill_kernel): a row is shared by a cluster of up to 8 blocks, so that the rows fill
//     the GPU; each block keeps its slice in registers (rows above 256 KB are streamed twice). The
//     blocks exchange (maximum, sum) pairs of their warps through distributed shared memory and join
//     them in a fixed order.
//
// All statistics are fp32. With c = log2(e) / tau and R the rounded c m of a maximum m, an exponent is
// c z - R in one rounding (fma): what R's rounding and c's are off cancels between a logit and the
// sum it is divided by, so nothing large is lost in log p - log q. ex2.approx is good to 2 units in
// the last place.
//
// Measured: 2048 rows of 131072 bf16, 64 entries: 252 us with the gradient (4.2 TB/s), 116 without (4.6);
// 1024 of 131072 fp32 239 and 98 (5.5); 2048 of 32000 bf16 70 and 44. No unit is near its limit there;
// 1024 entries a row, which one warp reads, take 574 and 530.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "lowp.cuh"
#include "tcgemm_host.cuh"

namespace bakron {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxK = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What exponents are taken against: R = fl(c m) of a maximum m (0 where nothing is finite). Where R is
// large, as with masks of the type's lowest value, its rounding is too, and differences from m are
// taken first instead.
struct Ref {
    float m, R, c;
    static __device__ __forceinline__ Ref of(float m, float c) {
        return Ref{m, m == kNegInf ? 0.f : __fmul_rn(m, c), c};
    }
    __device__ __forceinline__ bool usual() const { return fabsf(R) < 65536.f; }
    // 2^(c (x - m))
    __device__ __forceinline__ float term(float x) const {
        return usual() ? ex2(fmaf(x, c, -R)) : ex2((x - m) * c);
    }
    template <int N>
    __device__ __forceinline__ void terms(float (&x)[N]) const {
        if (usual()) {
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = ex2(fmaf(x[k], c, -R));
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = ex2((x[k] - m) * c);
        }
    }
    // the factor that brings a sum taken against m2 here; a sum without a finite element (0 or
    // NaN) stays what it is
    __device__ __forceinline__ float carry(float m2) const {
        if (m2 == kNegInf) return 1.f;
        const Ref o = of(m2, c);
        return usual() ? ex2(o.usual() ? o.R - R : fmaf(m2, c, -R))
                       : ex2(o.usual() ? fmaf(-m, c, o.R) : (m2 - m) * c);
    }
    // (x - m) / tau
    __device__ __forceinline__ float scaled(float x) const {
        return (usual() ? fmaf(x, c, -R) : (x - m) * c) * kLn2;
    }
    __device__ __forceinline__ float own(float inv_tau) const { return usual() ? R * kLn2 : m * inv_tau; }
};

struct Teacher {
    const void* idx; int idx64; const void* t; int td; int k;
    const float* lse; const float* w; float inv_tau;
};

__device__ __forceinline__ long long index_at(const Teacher& T, size_t e) {
    return T.idx64 ? static_cast<const long long*>(T.idx)[e] : static_cast<const int*>(T.idx)[e];
}
__device__ __forceinline__ float logit_at(const Teacher& T, size_t e) {
    if (T.td == BAKRON_F32) return static_cast<const float*>(T.t)[e];
    if (T.td == BAKRON_F16) return to_f32(static_cast<const __half*>(T.t)[e]);
    return to_f32(static_cast<const __nv_bfloat16*>(T.t)[e]);
}

// Over a warp, in a fixed order; every lane gets them.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// What is kept of a teacher's list: p, log p, the student's logits, the indices (-1: absent; padded
// to whole int4s), a table to find indices that stand there twice (lists above 32 entries), sum p.
struct List {
    float *p, *lp, *zt; int *at, *seen; float* mass; int* twice;
};
// Slots of the table: a power of two, twice the list's length or more; none for short lists.
__host__ __device__ inline int table_slots(int k) {
    int n = 64;
    while (n < 2 * k) n *= 2;
    return k > 32 ? n : 0;
}

// A row's list, by one warp.
template <class X>
__device__ __forceinline__ void read_list(const Teacher& T, const X* z, int row, int V,
                                          const List& L, int* status) {
    const int lane = threadIdx.x & 31, slots = table_slots(T.k);
    for (int e = lane; e < slots; e += 32) L.seen[e] = -1;
    __syncwarp();
    float tmax = kNegInf;
    bool dup = false;
    // four entries a lane at once: their loads, then the loads that these lead to
    for (int j0 = lane; j0 - lane < T.k; j0 += 128) {
        int here[4];
        float t[4], x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + 32 * u;
            here[u] = -1, t[u] = kNegInf;
            if (j < T.k) {
                const size_t e = (size_t)row * T.k + j;
                const long long i = index_at(T, e);
                t[u] = logit_at(T, e);
                if (i >= V) set_status(status, BAKRON_ERR_INVALID_ARG);
                if (i >= 0 && i < V && t[u] != kNegInf) here[u] = (int)i;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = here[u] >= 0 ? to_f32(z[here[u]]) : 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + 32 * u;
            if (j < T.k) L.lp[j] = t[u], L.zt[j] = x[u];
            if (j < (T.k + 3) / 4 * 4) L.at[j] = here[u];
            if (here[u] >= 0) tmax = fmaxf(tmax, t[u]);
            if (T.k <= 32) {
                const unsigned same = __match_any_sync(0xffffffffu, here[u]);   // by every lane
                dup |= here[u] >= 0 && __popc(same) > 1;
            } else if (here[u] >= 0) {
                unsigned h = ((unsigned)here[u] * 2654435761u >> 16) & (slots - 1);
                for (int step = 0; step < slots; ++step, h = (h + 1) & (slots - 1)) {
                    const int was = atomicCAS(&L.seen[h], -1, here[u]);
                    dup |= was == here[u];
                    if (was == -1 || was == here[u]) break;
                }
            }
        }
    }
    __syncwarp();
    float tl = 0.f;      // log p_j = (t_j - tmax) / tau - tl
    if (T.lse) {
        tmax = 0.f;
        tl = T.lse[row];
    } else {
        tmax = warp_max(tmax);
        float sum = 0.f;
        for (int j = lane; j < T.k; j += 32)
            if (L.at[j] >= 0) sum += expf((L.lp[j] - tmax) * T.inv_tau);
        tl = logf(warp_sum(sum));
    }
    float mass = 0.f;
    for (int j = lane; j < T.k; j += 32) {
        float pj = 0.f;
        if (L.at[j] >= 0) {
            L.lp[j] = (L.lp[j] - tmax) * T.inv_tau - tl;
            pj = expf(L.lp[j]);
        }
        L.p[j] = pj;
        mass += pj;
    }
    mass = warp_sum(mass);
    dup = __any_sync(0xffffffffu, dup);
    if (lane == 0) *L.mass = mass, *L.twice = dup;
}

// The loss of a row, by one warp: log q = (z - m) / tau - l.
__device__ __forceinline__ float list_loss(const Teacher& T, const List& L, const Ref& ref, float l) {
    float kl = 0.f;
    for (int j = threadIdx.x & 31; j < T.k; j += 32)
        if (L.p[j] != 0.f) kl += L.p[j] * (L.lp[j] - (ref.scaled(L.zt[j]) - l));
    return warp_sum(kl);
}

// Sum of p over all entries of entry j's index, in the list's order.
__device__ __forceinline__ float list_p(const Teacher& T, const List& L, int j) {
    if (!*L.twice) return L.p[j];
    const int i = L.at[j];
    float pj = 0.f;
    for (int k = 0; k < T.k; k += 4) {
        const int4 a = *reinterpret_cast<const int4*>(L.at + k);
        if (a.x == i) pj += L.p[k];
        if (a.y == i) pj += L.p[k + 1];
        if (a.z == i) pj += L.p[k + 2];
        if (a.w == i) pj += L.p[k + 3];
    }
    return pj;
}

// Joins the (maximum, sum) pairs of a block's or cluster's warps, every warp for itself and all
// alike.
__device__ __forceinline__ Ref join_pairs(const float2* pairs, int count, float c, float& s) {
    const int lane = threadIdx.x & 31;
    float m = kNegInf;
    for (int k = lane; k < count; k += 32) m = fmaxf(m, pairs[k].x);
    const Ref ref = Ref::of(warp_max(m), c);
    s = 0.f;
    for (int k = lane; k < count; k += 32) s += pairs[k].y * ref.carry(pairs[k].x);
    s = warp_sum(s);
    if (fabsf(ref.m) == INFINITY) s = NAN;      // +inf, or nothing but -inf
    return ref;
}

// How a row lies to 16-byte boundaries: `head` elements, `body` vectors, `rest` elements.
template <class X> struct Span {
    int head, body, rest;
    __device__ __forceinline__ Span(const X* z, int V) {
        head = min(V, (int)((16 - reinterpret_cast<uintptr_t>(z) % 16) % 16 / sizeof(X)));
        body = (V - head) / Vec<X>::N;
        rest = V - head - body * Vec<X>::N;
    }
    // the element outside the vectors that thread tid takes, or -1
    __device__ __forceinline__ int extra(int tid, int V) const {
        return tid < head ? tid : tid >= 32 && tid < 32 + rest ? V - rest + tid - 32 : -1;
    }
};

// NV: 16-byte vectors that a thread holds (LOOP: of one round of the stream).
template <class X, int NV, bool LOOP>
__global__ void __launch_bounds__(kThreads, 4)
distill_kernel(const X* z, int V, int64_t ld, const Teacher T, float* __restrict__ loss,
               float* __restrict__ lse, X* dz, int64_t ldd, int* __restrict__ status) {
    constexpr int N = Vec<X>::N;
    __shared__ float mass_of_list;
    __shared__ int twice;
    __shared__ int seen[2 * kMaxK];
    __shared__ float2 pairs[8 * kWarps];              // (maximum, sum) of the cluster's warps
    __shared__ float p[kMaxK], lp[kMaxK], zt[kMaxK];
    __shared__ __align__(16) int at[kMaxK];
    const List L{p, lp, zt, at, seen, &mass_of_list, &twice};
    cg::cluster_group cluster = cg::this_cluster();
    const int ck = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = blockIdx.x / ck, tid = threadIdx.x;
    const float w = T.w ? T.w[row] : 1.f;
    z += (int64_t)row * ld;
    if (dz) dz += (int64_t)row * ldd;

    // The row: `head` elements up to a 16-byte boundary, `body` vectors, the rest. The blocks
    // share the vectors; head and rest (16 elements at most) are the first block's, one a thread.
    const Span<X> S(z, V);
    const int head = S.head, body = S.body, rest = S.rest;
    const int v0 = (int)((long long)body * rank / ck), v1 = (int)((long long)body * (rank + 1) / ck);
    const int extra = rank == 0 ? S.extra(tid, V) : -1;
    const uint4* zv = reinterpret_cast<const uint4*>(z + head);
    // the gradient's row may lie otherwise to the boundaries: element by element then
    const bool wide = reinterpret_cast<uintptr_t>(dz + head) % 16 == 0;

    if (w == 0.f) {
        if (rank == 0 && tid == 0) loss[row] = 0.f, lse[row] = 0.f;
        if (dz) {
            if (extra >= 0) from_f32(0.f, dz[extra]);
            for (int i = v0 + tid; i < v1; i += kThreads) {
                if (wide) {
                    reinterpret_cast<uint4*>(dz + head)[i] = make_uint4(0, 0, 0, 0);
                } else {
#pragma unroll
                    for (int c = 0; c < N; ++c) from_f32(0.f, dz[head + (int64_t)i * N + c]);
                }
            }
        }
        return;
    }

    // the slice is on its way before the teacher's list is looked at
    uint4 v[NV];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int i = base + u * kThreads + tid;
            v[u] = i < v1 ? zv[i] : Vec<X>::fill_low();
        }
    };
    load(v0);
    const float zx = extra >= 0 ? to_f32(z[extra]) : kNegInf;
    if (ck > 1) cluster.barrier_arrive();        // (every block has begun: see the exchange)

    // The teacher's list, by the last warp while the slice arrives; the first block needs it for the
    // loss, the others for their part of the gradient.
    const bool list = rank == 0 || dz;
    const int lane = tid & 31;
    if (list && tid >= kThreads - 32)
        read_list<X>(T, z, row, V, L, status);

    // the slice's maximum and sum, warp by warp
    const float c = T.inv_tau * kLog2e;
    float m = zx, s = 0.f;
    auto thread_max = [&] {
        uint4 b = Vec<X>::fill_low();
#pragma unroll
        for (int u = 0; u < NV; ++u) b = Vec<X>::top(b, v[u]);
        return Vec<X>::most(b);
    };
    auto thread_sum = [&](const Ref& ref, int base) {
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        if (ref.usual()) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                float f[N];
                Vec<X>::get(v[u], f);
#pragma unroll
                for (int k = 0; k < N; ++k) part[k % 4] += ex2(fmaf(f[k], c, -ref.R));
            }
        } else {        // from memory again: no second copy of the loop over the registers
            for (int i = base + tid; i < min(v1, base + NV * kThreads); i += kThreads) {
                float f[N];
                Vec<X>::get(zv[i], f);
#pragma unroll
                for (int k = 0; k < N; ++k) part[0] += ex2((f[k] - ref.m) * c);
            }
        }
        return (part[0] + part[1]) + (part[2] + part[3]);
    };
    if constexpr (!LOOP) {
        m = warp_max(fmaxf(m, thread_max()));
        s = thread_sum(Ref::of(m, c), v0);
        if (extra >= 0) s += Ref::of(m, c).term(zx);
    } else {
        m = warp_max(m);
        if (extra >= 0) s = Ref::of(m, c).term(zx);
        for (int base = v0;;) {
            const float top = fmaxf(m, warp_max(thread_max()));
            if (top > m) s *= Ref::of(top, c).carry(m), m = top;
            s += thread_sum(Ref::of(m, c), base);
            base += NV * kThreads;
            if (base >= v1) break;
            load(base);
        }
    }
    s = warp_sum(s);
    if (ck > 1) {
        cluster.barrier_wait();
        if ((tid & 31) < ck)
            cluster.map_shared_rank(pairs, tid & 31)[rank * kWarps + tid / 32] = make_float2(m, s);
        cluster.sync();
    } else {
        if ((tid & 31) == 0) pairs[tid / 32] = make_float2(m, s);
        __syncthreads();
    }
    const Ref ref = join_pairs(pairs, ck * kWarps, c, s);
    if (rank == 0 && tid >= kThreads - 32) {
        const float l = logf(s);
        const float kl = list_loss(T, L, ref, l);
        if (lane == 0) loss[row] = w * kl, lse[row] = ref.own(T.inv_tau) + l;
    }
    if (!dz) return;

    // the gradient: every element, then those of the list once more (from the packed values: the
    // unpacked ones would take twice the registers all the way)
#pragma unroll
    for (int u = 0; u < NV; ++u)
        asm volatile("" : "+r"(v[u].x), "+r"(v[u].y), "+r"(v[u].z), "+r"(v[u].w));
    const float f = w * T.inv_tau, mass = mass_of_list;
    const bool none = mass == 0.f;
    const float fq = none ? 0.f : f * mass / s;
    if (extra >= 0) from_f32(none ? 0.f : fq * ref.term(zx), dz[extra]);
    const auto put = [&](int i, const float (&x)[N]) {
        if (wide) {
            reinterpret_cast<uint4*>(dz + head)[i] = Vec<X>::put(x);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) from_f32(x[k], dz[head + (int64_t)i * N + k]);
        }
    };
    if (none || !ref.usual()) {
        for (int i = v0 + tid; i < v1; i += kThreads) {
            float x[N];
            Vec<X>::get(zv[i], x);
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = none ? 0.f : fq * ex2((x[k] - ref.m) * c);
            put(i, x);
        }
    } else {
        for (int base = v0; base < v1; base += NV * kThreads) {
            if (LOOP) load(base);
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int i = base + u * kThreads + tid;
                if (i >= v1) break;
                float x[N];
                Vec<X>::get(v[u], x);
#pragma unroll
                for (int k = 0; k < N; ++k) x[k] = fq * ex2(fmaf(x[k], c, -ref.R));
                put(i, x);
            }
        }
    }
    if (none) return;
    __syncthreads();
    for (int j = tid; j < T.k; j += kThreads) {
        const int i = at[j];
        if (i < 0) continue;
        const int vec = i < head || i >= V - rest ? -1 : (i - head) / N;
        if (vec < 0 ? rank != 0 : vec < v0 || vec >= v1) continue;
        from_f32(fq * ref.term(zt[j]) - f * list_p(T, L, j), dz[i]);
    }
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Blocks that go from row to row: DATA threads and a warp for the lists. `keep`: vectors of a row
// that a thread keeps in shared memory; the next kRegs are kept in registers, others are streamed.
template <class X, int DATA, bool GRAD>
__global__ void __launch_bounds__(DATA + 32, 1024 / DATA)
distill_rows_kernel(const X* z0, int rows, int V, int64_t ld, const Teacher T,
                    float* __restrict__ loss, float* __restrict__ lse, X* dz0, int64_t ldd,
                    int* __restrict__ status, int keep) {
    constexpr int N = Vec<X>::N, ALL = DATA + 32;
    constexpr int kRegs = DATA == 992 ? 4 : 0, kHeld = kRegs > 0 ? kRegs : 1;
    enum { kData = 1, kListReady = 2, kListFree = 4 };      // barriers (the last two: one a buffer)
    extern __shared__ __align__(16) char smem[];
    __shared__ float2 pairs[2][DATA / 32];
    __shared__ float mass_of_list[2];
    __shared__ int twice[2];
    const int tid = threadIdx.x, lane = tid & 31, step = gridDim.x;
    const int k4 = (T.k + 3) / 4 * 4;
    float* lists = reinterpret_cast<float*>(smem + (size_t)keep * DATA * 16);
    const auto list = [&](int b) {
        float* l = lists + b * 4 * k4;
        return List{l, l + k4, l + 2 * k4, reinterpret_cast<int*>(l + 3 * k4),
                    reinterpret_cast<int*>(lists + 8 * k4), &mass_of_list[b], &twice[b]};
    };

    if (tid >= DATA) {
        for (int row = blockIdx.x, it = 0; row < rows; row += step, ++it) {
            if (it >= 2) bar_sync(kListFree + (it & 1), ALL);
            if (!T.w || T.w[row] != 0.f)
                read_list<X>(T, z0 + (int64_t)row * ld, row, V, list(it & 1), status);
            __syncwarp();
            bar_arrive(kListReady + (it & 1), ALL);
        }
        return;
    }

    const float c = T.inv_tau * kLog2e;
    uint4* slot = reinterpret_cast<uint4*>(smem) + tid;
    const uint32_t slot32 = (uint32_t)__cvta_generic_to_shared(slot);
    const auto weight = [&](int row) { return row < rows ? T.w ? T.w[row] : 1.f : 0.f; };
    // copies of the vectors that are kept of the row to come, slot by slot
    // Rows that are whole vectors apart lie alike to the boundaries.
    struct Next { const uint4* v; int body; };
    const bool alike = ld * (int64_t)sizeof(X) % 16 == 0;
    const Span<X> S0(z0, V);
    const auto next_row = [&](const X* z, float w) {
        const Span<X> S = alike ? S0 : Span<X>(z, V);
        return Next{reinterpret_cast<const uint4*>(z + S.head) + tid, w != 0.f ? S.body : 0};
    };
    const auto copy = [&](const Next& nx, int u) {
        if (u * DATA + tid < nx.body)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot32 + u * DATA * 16),
                         "l"(nx.v + u * DATA)
                         : "memory");
    };
    // They are made and waited for in groups of four slots, `groups` a row (empty ones included), so
    // that what is pending can be counted.
    const int groups = (keep + 3) / 4;
    unsigned long long once;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    const auto copy_group = [&](const Next& nx, int q) {
        if (4 * q + 4 <= keep && (4 * q + 4) * DATA <= nx.body) {
            const uint4* src = nx.v + 4 * q * DATA;
            const uint32_t dst = slot32 + 4 * q * DATA * 16;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst + u * DATA * 16),
                             "l"(src + u * DATA), "l"(once)
                             : "memory");
        } else {
            for (int u = 4 * q; u < min(4 * q + 4, keep); ++u) copy(nx, u);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto wait = [](int pending) {
        switch (pending) {
            case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
            case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
            case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
            default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        }
    };

    float w = weight(blockIdx.x);
    const X* z = z0 + (int64_t)blockIdx.x * ld;
    X* dz = GRAD ? dz0 + (int64_t)blockIdx.x * ldd : nullptr;
    {
        const Next first_row = next_row(z, w);
        for (int q = 0; q < groups; ++q) copy_group(first_row, q);
    }
    for (int row = blockIdx.x, it = 0; row < rows; row += step, ++it) {
        const int b = it & 1;
        const Span<X> S = alike ? S0 : Span<X>(z, V);
        const int extra = S.extra(tid, V);
        const uint4* zv = reinterpret_cast<const uint4*>(z + S.head);
        uint4* dv = reinterpret_cast<uint4*>(dz + S.head);
        const bool wide = reinterpret_cast<uintptr_t>(dz + S.head) % 16 == 0;
        const float w_next = weight(row + step);
        const Next next = next_row(z + (int64_t)step * ld, w_next);
        const auto put = [&](int i, const float (&x)[N]) {
            if (wide) {
                __stcs(dv + i, Vec<X>::put(x));
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) from_f32(x[k], dz[S.head + (int64_t)i * N + k]);
            }
        };
        const auto put_zeros = [&] {
            const float zero[N] = {};
            if (extra >= 0) from_f32(0.f, dz[extra]);
            for (int i = tid; i < S.body; i += DATA) put(i, zero);
        };
        // vectors of this thread behind those that are kept: f(index, four of them) as long as every
        // thread has four, then f(index, one)
        const auto stream = [&](auto f) {
            for (int base = (keep + kRegs) * DATA; base < S.body; base += 4 * DATA) {
                const uint4* from = zv + base + tid;
                if (base + 4 * DATA <= S.body) {
                    uint4 v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[u] = from[u * DATA];
                    f(base + tid, v);
                } else {
                    for (int i = base + tid; i < S.body; i += DATA) {
                        const uint4 v[1] = {zv[i]};
                        f(i, v);
                    }
                }
            }
        };

        if (w == 0.f) {
            for (int q = 0; q < groups; ++q) copy_group(next, q);
            bar_sync(kListReady + b, ALL);
            if (tid == 0) loss[row] = 0.f, lse[row] = 0.f;
            if (GRAD) put_zeros();
        } else {
            // this thread's maximum m and sum
            const float zx = extra >= 0 ? to_f32(z[extra]) : kNegInf;
            float m = kNegInf, s = 0.f;
            const auto add = [&](const auto& v) {
                constexpr int count = sizeof(v) / sizeof(uint4);
                uint4 top = v[0];
#pragma unroll
                for (int u = 1; u < count; ++u) top = Vec<X>::top(top, v[u]);
                const float a = fmaxf(m, Vec<X>::most(top));
                float f[N];
                if (a > m) s *= Ref::of(a, c).carry(m), m = a;
                const Ref own = Ref::of(m, c);
                float part[2] = {0.f, 0.f};
#pragma unroll
                for (int u = 0; u < count; ++u) {
                    Vec<X>::get(v[u], f);
                    own.terms(f);
#pragma unroll
                    for (int k = 0; k < N; ++k) part[k % 2] += f[k];
                }
                s += part[0] + part[1];
            };
            uint4 held[kHeld];
            const bool hold = kRegs > 0 && keep * DATA < S.body;
            if (hold) {
#pragma unroll
                for (int u = 0; u < kRegs; ++u) {
                    const int i = (keep + u) * DATA + tid;
                    held[u] = i < S.body ? zv[i] : Vec<X>::fill_low();
                }
            }
            stream([&](int, const auto& v) { add(v); });
            for (int q = 0; q < groups; ++q) {
                wait(GRAD ? groups - 1 - q : groups - 1);
                // a whole group, one with most of its vectors (the others count as -inf), or the
                // one or two that are left
                const int have = min(4 * q + 4, keep);
                if (have * DATA <= S.body && have == 4 * q + 4) {
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = slot[(4 * q + k) * DATA];
                    add(v);
                } else if (min(have * DATA, S.body) > (4 * q + 2) * DATA) {
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int u = 4 * q + k;
                        v[k] = u < keep && u * DATA + tid < S.body ? slot[u * DATA]
                                                                   : Vec<X>::fill_low();
                    }
                    add(v);
                } else {
                    for (int u = 4 * q; u < have && u * DATA + tid < S.body; ++u) {
                        const uint4 v[1] = {slot[u * DATA]};
                        add(v);
                    }
                }
                if (!GRAD) copy_group(next, q);
            }
            if (hold) add(held);
            const float mw = warp_max(fmaxf(m, zx));
            s *= Ref::of(mw, c).carry(m);
            if (extra >= 0) s += Ref::of(mw, c).term(zx);
            s = warp_sum(s);
            if (lane == 0) pairs[b][tid / 32] = make_float2(mw, s);
            bar_sync(kData, DATA);
            const Ref ref = join_pairs(pairs[b], DATA / 32, c, s);
            bar_sync(kListReady + b, ALL);
            const List L = list(b);
            if (tid < 32) {
                const float l = logf(s), kl = list_loss(T, L, ref, l);
                if (tid == 0) loss[row] = w * kl, lse[row] = ref.own(T.inv_tau) + l;
            }
            if (GRAD) {
                const float f = w * T.inv_tau, mass = *L.mass;
                const float fq = f * mass / s;
                const auto write = [&](int i, const uint4& v) {
                    float x[N];
                    Vec<X>::get(v, x);
                    ref.terms(x);
#pragma unroll
                    for (int k = 0; k < N; ++k) x[k] *= fq;
                    put(i, x);
                };
                const bool plain = wide && ref.usual() && mass != 0.f;
                // four whole rounds of plain vectors
                const auto write4 = [&](int i, const uint4 (&v)[4]) {
                    uint4* to = dv + i;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float x[N];
                        Vec<X>::get(v[u], x);
#pragma unroll
                        for (int k = 0; k < N; ++k) x[k] = fq * ex2(fmaf(x[k], c, -ref.R));
                        __stcs(to + u * DATA, Vec<X>::put(x));
                    }
                };
                for (int q = 0; q < groups; ++q) {
                    if (plain && 4 * q + 4 <= keep && (4 * q + 4) * DATA <= S.body) {
                        uint4 v[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) v[u] = slot[(4 * q + u) * DATA];
                        write4(4 * q * DATA + tid, v);
                    } else if (mass != 0.f) {
                        for (int u = 4 * q; u < min(4 * q + 4, keep); ++u)
                            if (u * DATA + tid < S.body) write(u * DATA + tid, slot[u * DATA]);
                    }
                    copy_group(next, q);
                }
                if (mass != 0.f) {
                    if (hold) {
#pragma unroll
                        for (int u = 0; u < kRegs; ++u) {
                            const int i = (keep + u) * DATA + tid;
                            if (i < S.body) write(i, held[u]);
                        }
                    }
                    stream([&](int i, const auto& v) {
                        constexpr int count = sizeof(v) / sizeof(uint4);
                        if constexpr (count == 4) {
                            if (plain) {
                                write4(i, v);
                                return;
                            }
                        }
#pragma unroll
                        for (int u = 0; u < count; ++u) write(i + u * DATA, v[u]);
                    });
                    if (extra >= 0) from_f32(fq * ref.term(zx), dz[extra]);
                    bar_sync(kData, DATA);
                    for (int j = tid; j < T.k; j += DATA)
                        if (L.at[j] >= 0)
                            from_f32(fq * ref.term(L.zt[j]) - f * list_p(T, L, j),
                                     dz[L.at[j]]);
                } else {
                    put_zeros();        // an empty list, whatever the logits are
                }
            }
        }
        if (row + 2 * (int64_t)step < rows) bar_arrive(kListFree + b, ALL);
        w = w_next, z += (int64_t)step * ld;
        if (GRAD) dz += (int64_t)step * ldd;
    }
}

template <class X, int NV, bool LOOP>
int launch(const X* z, int rows, int V, int64_t ld, const Teacher& T, float* loss, float* lse, X* dz,
           int64_t ldd, int* status, int ck, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * ck);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ck;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, distill_kernel<X, NV, LOOP>, z, V, ld, T, loss,
                                             lse, dz, ldd, status);
    count_launches(1);
    return cuda_err(e);
}

// What the blocks of an SM share; one block takes less (at most 512 bytes of static arrays beside it).
constexpr size_t kRowsSmem = 226 * 1024;

template <class X, int DATA>
int launch_rows(const X* z, int rows, int V, int64_t ld, const Teacher& T, float* loss, float* lse,
                X* dz, int64_t ldd, int* status, int sms, cudaStream_t st) {
    constexpr int blocks = 1024 / DATA;         // of an SM (1 of 992)
    const size_t lists = (size_t)32 * ((T.k + 3) / 4 * 4) + (size_t)table_slots(T.k) * 4;
    const size_t room = kRowsSmem / blocks - 1024 - 512;     // reserved, and the static arrays
    const size_t vec = (size_t)DATA * 16;
    size_t keep = room > lists ? (room - lists) / vec : 0;
    keep = std::min({keep, (size_t)16, ((size_t)V / Vec<X>::N + DATA - 1) / DATA});
    // whole groups of four, unless the row ends within them
    if (keep * DATA < (size_t)V / Vec<X>::N) keep -= keep % 4;
    const size_t smem = keep * vec + lists;
    auto kern = dz ? distill_rows_kernel<X, DATA, true> : distill_rows_kernel<X, DATA, false>;
    if (smem > kRowsSmem || !allow_smem<kRowsSmem>(kern)) return BAKRON_ERR_CUDA;
    kern<<<std::min(rows, blocks * sms), DATA + 32, smem, st>>>(z, rows, V, ld, T, loss, lse, dz, ldd,
                                                                status, (int)keep);
    count_launches(1);
    return cuda_err(cudaGetLastError());
}

template <int D>
int plan(const void* z_, int rows, int V, int64_t ld, const Teacher& T, float* loss, float* lse,
         void* dz_, int64_t ldd, int* status, cudaStream_t st) {
    using X = typename Elem<D>::T;
    const X* z = static_cast<const X*>(z_);
    X* dz = static_cast<X*>(dz_);
    const int sms = tc::sm_count();
    if (sms <= 0) return BAKRON_ERR_CUDA;
    // Many rows: eight blocks of 128 threads an SM up to 24 KB a row, then two of 512, and one of 992
    // above 384 KB, where two rows an SM would read most of themselves twice (measured when chosen,
    // with the gradient, 512 / 992 threads: 260 / 280 us for 2048 rows of 256 KB, 293 / 239 us for
    // 1024 of 512 KB; four blocks of 256 for 64 KB took 76 us, two of 512 take 72).
    if (rows >= 2 * sms) {
        const size_t row = (size_t)V * sizeof(X);
        if (row <= 24 * 1024)
            return launch_rows<X, 128>(z, rows, V, ld, T, loss, lse, dz, ldd, status, sms, st);
        if (row <= 384 * 1024)
            return launch_rows<X, 512>(z, rows, V, ld, T, loss, lse, dz, ldd, status, sms, st);
        return launch_rows<X, 992>(z, rows, V, ld, T, loss, lse, dz, ldd, status, sms, st);
    }
    // Few rows. Blocks a row: as many as keep its slices within 8 vectors a thread or fill the GPU
    // (four blocks an SM), as long as a slice has a vector for every thread.
    const int vecs = V / Vec<X>::N;
    int ck = 1;
    while (ck < 8 && vecs > ck * 8 * kThreads) ck *= 2;
    while (ck < 8 && (long long)rows * ck * 2 <= 4 * sms && vecs > ck * kThreads) ck *= 2;
    if ((long long)rows * ck > INT32_MAX) return BAKRON_ERR_INVALID_ARG;
    const int nv = (vecs + ck * kThreads - 1) / (ck * kThreads);
    // a slice is ceil(vecs / ck) vectors at most
    if (nv <= 1) return launch<X, 1, false>(z, rows, V, ld, T, loss, lse, dz, ldd, status, ck, st);
    if (nv <= 2) return launch<X, 2, false>(z, rows, V, ld, T, loss, lse, dz, ldd, status, ck, st);
    if (nv <= 4) return launch<X, 4, false>(z, rows, V, ld, T, loss, lse, dz, ldd, status, ck, st);
    if (nv <= 8) return launch<X, 8, false>(z, rows, V, ld, T, loss, lse, dz, ldd, status, ck, st);
    return launch<X, 4, true>(z, rows, V, ld, T, loss, lse, dz, ldd, status, ck, st);
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" int bakron_distill(const void* logits, int dtype, int rows, int vocab, int64_t ld,
                              const void* top_idx, int idx_dtype, const void* top_logits,
                              int top_dtype, int k, const float* teacher_lse,
                              const float* row_weights, float temperature, float* loss,
                              float* lse, void* dlogits, int64_t ldd, int* dev_status,
                              void* stream) {
    if (!float_dtype(dtype) || !float_dtype(top_dtype) ||
        (idx_dtype != BAKRON_I32 && idx_dtype != BAKRON_I64) || rows < 0 || rows > (1 << 30) ||
        vocab < 1 ||
        ld < vocab || (dlogits && ldd < vocab) || (dlogits == logits && dlogits && ldd != ld) ||
        k < 1 || k > kMaxK || !(temperature > 0.f) || !std::isfinite(temperature) ||
        !std::isfinite(1.f / temperature))
        return BAKRON_ERR_INVALID_ARG;
    if (rows == 0) return BAKRON_OK;
    if (!logits || !top_idx || !top_logits || !loss || !lse || !dev_status ||
        !aligned_to(logits, dtype_bytes(dtype)) || !aligned_to(dlogits, dtype_bytes(dtype)) ||
        !aligned_to(top_idx, dtype_bytes(idx_dtype)) ||
        !aligned_to(top_logits, dtype_bytes(top_dtype)))
        return BAKRON_ERR_INVALID_ARG;
    const Teacher T{top_idx, idx_dtype == BAKRON_I64, top_logits, top_dtype, k, teacher_lse,
                    row_weights, 1.f / temperature};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case BAKRON_F32:
            return plan<BAKRON_F32>(logits, rows, vocab, ld, T, loss, lse, dlogits, ldd, dev_status,
                                    st);
        case BAKRON_F16:
            return plan<BAKRON_F16>(logits, rows, vocab, ld, T, loss, lse, dlogits, ldd, dev_status,
                                    st);
        default:
            return plan<BAKRON_BF16>(logits, rows, vocab, ld, T, loss, lse, dlogits, ldd,
                                     dev_status, st);
    }
}
