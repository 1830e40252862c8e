// Verification of drafted tokens against the target's probabilities from
// given uniform numbers (tq_verify_draft).
//
// Nodes of one sequence are in drafting order, node 0 the last token that is
// already certain; row n of `target` is the target's distribution after node
// n, row n of `draft` the one that n's children were drawn from.  From node
// n, with w = target[n], the children c are tried in order:
//     accepted when u[c] * q(x_c) < w(x_c): go on from c;
//     else w <- max(w - q, 0) / sum max(w - q, 0)    (draft given), or
//          w(x_c) <- 0, the threshold u * (1 - what was removed)   (none).
// After the last one the next token is the first index whose running sum of w
// passes r times the sum.  After j rejections w = max(a p - b q, 0) for two
// scalars a, b, so no row is ever written.  Everything is fp64: an index then
// depends on the order of a sum with a probability of about 1e-13.
//
// Bound: the rows the last token is drawn from are read once (HBM; for one
// sequence, latency: tokens -> their probabilities -> the row).  A sequence's
// row is cut into tiles of TILE elements, one workgroup each; every workgroup
// walks the drafted nodes itself (a few values in LDS), sums its tile, and
// the last one to finish finds the tile that holds the threshold and the
// element in it.  Trees drafted with probabilities need whole-row sums during
// the walk and run as one workgroup per sequence instead.
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int TILE = 2048;
constexpr int MAX_NODES = 1024;

template <int DT> __device__ __forceinline__ double prob(const void *p, int64_t i)
{
    if constexpr (DT == TQ_F32)
        return (double)((const float *)p)[i];
    else if constexpr (DT == TQ_BF16)
        return (double)__builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
    else
        return (double)f16_bits_to_f32(((const uint16_t *)p)[i]);
}

__device__ __forceinline__ double positive(double x) { return x > 0.0 ? x : 0.0; }

// What the walk needs of each node, and its result.
struct Walk {
    int parent[MAX_NODES], token[MAX_NODES];
    float u[MAX_NODES];
    double p[MAX_NODES], q[MAX_NODES];
    int path[MAX_NODES];                         // accepted nodes, then the rejected ones
};

struct Found {
    int taken, rejected, node;                   // path[0..taken), then `rejected` more
    double a, b;                                 // last token from max(a p - b q, 0), ...
    double a0, b0;                               // ... or, where that is all zero, this one
};

struct Seq {
    int64_t n0;
    int T;
};

__device__ __forceinline__ Seq seq_of(const VerifyArgs &a, int b)
{
    const int64_t s0 = min(max((int64_t)a.starts[b], (int64_t)0), a.nodes);
    const int64_t s1 = min((int64_t)a.starts[b + 1], a.nodes);
    return {s0, (int)min(max(s1 - s0, (int64_t)0), (int64_t)a.width)};
}

template <int DT>
__device__ __forceinline__ void load_nodes(const VerifyArgs &a, const Seq &s, Walk &w, int tid,
                                           int threads)
{
    for (int i = tid; i < s.T; i += threads) {
        const int par = a.parents ? a.parents[s.n0 + i] : i - 1;
        const int64_t x = a.tokens[s.n0 + i];
        // a child after its parent and inside the vocabulary, or never accepted
        const bool ok = i > 0 && par >= 0 && par < i && x >= 0 && x < a.vocab;
        w.parent[i] = i > 0 && par >= 0 && par < i ? par : -1;
        w.token[i] = (int)(ok ? x : -1);
        w.u[i] = a.u[s.n0 + i];
        w.p[i] = ok ? positive(prob<DT>(a.target, (s.n0 + par) * a.target_stride + x)) : 0.0;
        w.q[i] = ok && a.draft ? prob<DT>(a.draft, (s.n0 + par) * a.draft_stride + x) : 0.0;
    }
}

// The walk.  row_sum(node, a, b): sum of max(a p - b q, 0), called only for a
// sibling after a rejection with draft probabilities given.  Without those one
// thread walks (`writer`) and reads path[] back; with them path[] is only
// written, so a whole workgroup may walk alike and join in row_sum.
template <typename F>
__device__ __forceinline__ Found walk(const VerifyArgs &a, const Seq &s, Walk &w, bool writer,
                                      F row_sum)
{
    Found f{0, 0, 0, 1.0, 0.0, 1.0, 0.0};
    double left = 1.0;
    bool pending = false;                        // the last rejection's sum is not taken yet
    for (int i = 1; i < s.T; i++) {
        if (w.parent[i] != f.node)
            continue;
        if (w.token[i] < 0)
            continue;
        bool good;
        double p = w.p[i];
        if (a.draft) {
            if (pending) {
                const double z = row_sum(f.node, f.a, f.b);
                if (z > 0.0) {
                    f.a /= z;
                    f.b /= z;
                } else {
                    f.a = f.a0;
                    f.b = f.b0;
                }
                pending = false;
            }
            good = (double)w.u[i] * w.q[i] < positive(f.a * p - f.b * w.q[i]);
        } else {
            // a sibling with the same token has taken its probability along
            for (int k = 0; k < f.rejected; k++)
                if (w.token[w.path[f.taken + k]] == w.token[i])
                    p = 0.0;
            good = p > 0.0 && (double)w.u[i] * left < p;
        }
        if (good) {
            f.node = i;
            if (writer)
                w.path[f.taken] = i;
            f.taken++;
            f.rejected = 0;
            f.a = f.a0 = 1.0;
            f.b = f.b0 = 0.0;
            left = 1.0;
        } else if (a.draft) {
            f.a0 = f.a;
            f.b0 = f.b;
            f.b += 1.0;
            pending = true;
        } else {
            if (writer)
                w.path[f.taken + f.rejected] = i;
            f.rejected++;
            left -= p;
        }
    }
    return f;
}

// Weight of vocabulary entry x at node row `row`, and the fallback's.
template <int DT>
__device__ __forceinline__ void weights(const VerifyArgs &a, const Walk &w, const Found &f,
                                        int64_t row, int64_t x, double &now, double &before)
{
    const double p = prob<DT>(a.target, row * a.target_stride + x);
    if (a.draft) {
        const double q = prob<DT>(a.draft, row * a.draft_stride + x);
        now = positive(f.a * p - f.b * q);
        before = positive(f.a0 * p - f.b0 * q);
    } else {
        now = positive(p);
        for (int k = 0; k < f.rejected; k++)
            if (w.token[w.path[f.taken + k]] == x)
                now = 0.0;
        before = 0.0;
    }
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        v += __shfl_xor(v, m);
    return v;
}

// The tile whose running sum passes the threshold, and the sum before it.
struct Place {
    int tile;
    double before;
};

// Looks for the element in tile `place.tile` (the first 256 threads) and
// writes the sequence's outputs.
template <int DT>
__device__ __forceinline__ void finish(const VerifyArgs &a, int b, const Seq &s, const Walk &w,
                                       const Found &f, bool use_before, const Place &place,
                                       double thr, double total, int *pick)
{
    __shared__ double part[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    constexpr int PER = TILE / 256;
    double v[PER], sum = 0.0;
    const int64_t x0 = (int64_t)place.tile * TILE + tid * PER;
    if (tid == 0) {
        pick[0] = 0x7fffffff;                    // first element past the threshold
        pick[1] = -1;                            // last element of positive weight
    }
#pragma unroll
    for (int e = 0; e < PER; e++) {
        double now = 0.0, before = 0.0;
        if (s.T > 0 && tid < 256 && x0 + e < a.vocab)
            weights<DT>(a, w, f, s.n0 + f.node, x0 + e, now, before);
        v[e] = use_before ? before : now;
        sum += v[e];
    }
    double run = sum;                            // inclusive over the wave's threads
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(run, m);
        if (lane >= m)
            run += o;
    }
    if (tid < 256 && lane == 63)
        part[wave] = run;
    __syncthreads();
    if (tid < 256 && total > 0.0) {
        double at = place.before + (run - sum);
        for (int k = 0; k < wave; k++)
            at += part[k];
        int hit = 0x7fffffff, last = -1;
#pragma unroll
        for (int e = 0; e < PER; e++) {
            at += v[e];
            if (v[e] > 0.0) {
                last = (int)(x0 + e);
                if (at > thr && hit == 0x7fffffff)
                    hit = last;
            }
        }
        if (hit != 0x7fffffff)
            atomicMin(&pick[0], hit);
        if (last >= 0)
            atomicMax(&pick[1], last);
    }
    __syncthreads();
    const int next = pick[0] != 0x7fffffff ? pick[0] : pick[1];
    for (int i = tid; i < a.width; i += blockDim.x) {
        const bool in = i < f.taken;
        a.out_nodes[(int64_t)b * a.width + i] = in ? w.path[i] : -1;
        a.out_tokens[(int64_t)b * a.width + i] =
            in ? w.token[w.path[i]] : (i == f.taken && s.T > 0 ? next : -1);
    }
    if (tid == 0)
        a.count[b] = f.taken;
}

// Running search over tile sums by one wave: lane k of a round holds tile
// base + k.  sums(i) gives tile i's sum.
template <typename F>
__device__ __forceinline__ Place find_tile(int tiles, double thr, F sums)
{
    const int lane = threadIdx.x & 63;
    double before = 0.0, last_before = 0.0;
    int last = 0;                                // last tile of positive sum
    for (int base = 0; base < tiles; base += 64) {
        const double v = base + lane < tiles ? sums(base + lane) : 0.0;
        double run = v;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double o = __shfl_up(run, m);
            if (lane >= m)
                run += o;
        }
        const double prev = before + (run - v);
        const uint64_t hit = __ballot(v > 0.0 && before + run > thr);
        if (hit) {
            const int k = __builtin_ctzll(hit);
            return {base + k, __shfl(prev, k)};
        }
        const uint64_t some = __ballot(v > 0.0);
        if (some) {
            const int k = 63 - __builtin_clzll(some);
            last = base + k;
            last_before = __shfl(prev, k);
        }
        before += __shfl(run, 63);
    }
    return {last, last_before};
}

// Chains, and trees without draft probabilities: one workgroup per (tile,
// sequence).
template <int DT>
__global__ __launch_bounds__(256) void k_verify(VerifyArgs a, int tiles, uint32_t *counters,
                                                double *sums)
{
    __shared__ Walk w;
    __shared__ double red[2][4];
    __shared__ int pick[2], last_flag;
    __shared__ Found found;
    __shared__ Place place;
    __shared__ double total_s;
    __shared__ int before_s;
    const int tile = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const Seq s = seq_of(a, b);
    load_nodes<DT>(a, s, w, tid, 256);
    __syncthreads();
    if (tid == 0)
        found = walk(a, s, w, true, [](int, double, double) { return 1.0; });
    __syncthreads();
    const Found f = found;

    double now = 0.0, before = 0.0;
    if (s.T > 0)
        for (int e = 0; e < TILE / 256; e++) {
            const int64_t x = (int64_t)tile * TILE + e * 256 + tid;
            if (x < a.vocab) {
                double n, o;
                weights<DT>(a, w, f, s.n0 + f.node, x, n, o);
                now += n;
                before += o;
            }
        }
    now = wave_sum(now);
    before = wave_sum(before);
    if ((tid & 63) == 0) {
        red[0][tid >> 6] = now;
        red[1][tid >> 6] = before;
    }
    __syncthreads();
    double *mine = sums + (int64_t)b * tiles * 2;
    if (tid == 0) {
        __hip_atomic_store(mine + 2 * tile, (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(mine + 2 * tile + 1, (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint32_t done = __hip_atomic_fetch_add(counters + b, 1u, __ATOMIC_ACQ_REL,
                                                     __HIP_MEMORY_SCOPE_AGENT);
        last_flag = done == (uint32_t)tiles - 1;
    }
    __syncthreads();
    if (!last_flag)
        return;
    auto sum_of = [&](int use, int i) {
        return __hip_atomic_load(mine + 2 * i + use, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    if (tid < 64) {
        double t0 = 0.0, t1 = 0.0;
        for (int i = tid; i < tiles; i += 64) {
            t0 += sum_of(0, i);
            t1 += sum_of(1, i);
        }
        t0 = wave_sum(t0);
        t1 = wave_sum(t1);
        const int use = t0 > 0.0 ? 0 : 1;
        const double total = use ? t1 : t0;
        const double thr = (double)a.r[b] * total;
        const Place at = find_tile(tiles, thr, [&](int i) { return sum_of(use, i); });
        if (tid == 0) {
            place = at;
            total_s = total;
            before_s = use;
            // zero again for the next call on this workspace
            __hip_atomic_store(counters + b, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    __syncthreads();
    finish<DT>(a, b, s, w, f, before_s != 0, place, (double)a.r[b] * total_s, total_s, pick);
}

// Trees with draft probabilities: one workgroup per sequence.
constexpr int TREE_THREADS = 1024;

template <int DT>
__global__ __launch_bounds__(TREE_THREADS) void k_verify_tree(VerifyArgs a, int tiles,
                                                              double *sums)
{
    __shared__ Walk w;
    __shared__ double red[2][TREE_THREADS / 64];
    __shared__ int pick[2];
    __shared__ Place place;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Seq s = seq_of(a, b);
    load_nodes<DT>(a, s, w, tid, TREE_THREADS);
    __syncthreads();
    auto row_sum = [&](int node, double fa, double fb) {
        double v = 0.0;
        const int64_t row = s.n0 + node;
        for (int64_t x = tid; x < a.vocab; x += TREE_THREADS)
            v += positive(fa * prob<DT>(a.target, row * a.target_stride + x) -
                          fb * prob<DT>(a.draft, row * a.draft_stride + x));
        v = wave_sum(v);
        __syncthreads();
        if (lane == 0)
            red[0][wave] = v;
        __syncthreads();
        double z = 0.0;
        for (int k = 0; k < TREE_THREADS / 64; k++)
            z += red[0][k];
        return z;
    };
    const Found f = walk(a, s, w, tid == 0, row_sum);
    __syncthreads();

    double *mine = sums + (int64_t)b * tiles * 2;
    double t0 = 0.0, t1 = 0.0;                   // the same in every lane of a wave
    for (int tile = wave; tile < tiles; tile += TREE_THREADS / 64) {
        double now = 0.0, before = 0.0;
        if (s.T > 0)
            for (int e = 0; e < TILE / 64; e++) {
                const int64_t x = (int64_t)tile * TILE + e * 64 + lane;
                if (x < a.vocab) {
                    double n, o;
                    weights<DT>(a, w, f, s.n0 + f.node, x, n, o);
                    now += n;
                    before += o;
                }
            }
        now = wave_sum(now);
        before = wave_sum(before);
        if (lane == 0) {
            mine[2 * tile] = now;
            mine[2 * tile + 1] = before;
        }
        t0 += now;
        t1 += before;
    }
    __syncthreads();
    if (lane == 0) {
        red[0][wave] = t0;
        red[1][wave] = t1;
    }
    __syncthreads();
    t0 = t1 = 0.0;
    for (int k = 0; k < TREE_THREADS / 64; k++) {
        t0 += red[0][k];
        t1 += red[1][k];
    }
    const int use = t0 > 0.0 ? 0 : 1;
    const double total = use ? t1 : t0;
    const double thr = (double)a.r[b] * total;
    if (tid < 64) {
        const Place at = find_tile(tiles, thr, [&](int i) { return mine[2 * i + use]; });
        if (tid == 0)
            place = at;
    }
    __syncthreads();
    finish<DT>(a, b, s, w, f, use != 0, place, thr, total, pick);
}

int tiles_of(int64_t vocab) { return (int)((vocab + TILE - 1) / TILE); }

template <int DT>
hipError_t launch_dt(const VerifyArgs &a, uint32_t *counters, double *sums, hipStream_t s)
{
    const int tiles = tiles_of(a.vocab);
    if (a.parents && a.draft) {
        k_verify_tree<DT><<<dim3((unsigned)a.batch), TREE_THREADS, 0, s>>>(a, tiles, sums);
    } else {
        k_verify<DT><<<dim3((unsigned)tiles, (unsigned)a.batch), 256, 0, s>>>(a, tiles, counters, sums);
    }
    return hipGetLastError();
}

}  // namespace

size_t verify_scratch_bytes(int64_t batch, int64_t vocab)
{
    return (size_t)batch * tiles_of(vocab) * 2 * sizeof(double);
}

hipError_t launch_verify(int dtype, const VerifyArgs &a, uint32_t *counters, void *scratch,
                         hipStream_t s)
{
    switch (dtype) {
    case TQ_F32: return launch_dt<TQ_F32>(a, counters, (double *)scratch, s);
    case TQ_BF16: return launch_dt<TQ_BF16>(a, counters, (double *)scratch, s);
    case TQ_F16: return launch_dt<TQ_F16>(a, counters, (double *)scratch, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace tq
