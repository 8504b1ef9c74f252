// Plan of a batch whose tokens belong to many adapters, on gfx950: a stable counting sort
// of the tokens by adapter and the work lists that the multi-adapter kernels walk. Made
// once for a batch and used by every projection of the model.
//
// One workgroup of 16 waves: each wave counts a contiguous span of tokens into its own row
// of an LDS histogram (64 tokens at a time; equal ids of a wave instruction are matched by
// ballots over the id's bits, so the lanes of one id take consecutive places and the sort
// is stable and the same on every run), the rows become start positions, and a second pass
// over the same span writes the order. Bound by latency: two passes over M ids.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "multi.h"

namespace qn {
namespace {

constexpr int kPlanWaves = 16;
constexpr int kPlanThreads = 64 * kPlanWaves;
constexpr int kKeys = kMultiMaxAdapters + 1;          // + the tokens without an adapter

struct PlanOut {
    int32_t *head, *order, *start, *first_item, *used;
    int2* tile;
    MultiItem* items;
};

// exclusive sum of v over the workgroup's threads; total in *sum
__device__ __forceinline__ int block_scan(int v, int* tmp, int* sum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                                   // tmp is free
    if (lane == 63) tmp[wave] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        if (w < wave) before += tmp[w];
        all += tmp[w];
    }
    *sum = all;
    return before + x - v;
}

// lanes with the same key as this one (keys < 2^11)
__device__ __forceinline__ unsigned long long same_key(int key, bool valid) {
    unsigned long long m = __ballot(valid);
#pragma unroll
    for (int b = 0; b < 11; ++b) {
        const unsigned long long set = __ballot((key >> b) & 1);
        m &= ((key >> b) & 1) ? set : ~set;
    }
    return m;
}

__global__ __launch_bounds__(kPlanThreads)
void multi_plan_kernel(const int32_t* __restrict__ ids, int M, int n, int max_items, PlanOut out) {
    __shared__ int hist[kPlanWaves * kKeys];
    __shared__ int ends[kMultiMaxAdapters];            // end position of each adapter in use
    __shared__ int tmp[kPlanWaves];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int keys = n + 1;
    for (int i = tid; i < kPlanWaves * keys; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
    const int span = ((M + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64;
    const int t0 = wave * span, t1 = min(M, t0 + span);
    int* row = hist + wave * keys;
    const unsigned long long below = (1ull << lane) - 1;
    for (int t = t0; t < t1; t += 64) {
        const bool ok = t + lane < t1;
        const int id = ok ? ids[t + lane] : -1;
        const int key = id >= 0 && id < n ? id : n;
        const unsigned long long same = same_key(key, ok);
        if (ok && (same & below) == 0) row[key] += __popcll(same);       // the first lane of each id
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");           // seen by the next one's
    }
    __syncthreads();
    // thread k < n: adapter k (n <= 1024 threads)
    int count = 0;
    if (tid < n)
        for (int w = 0; w < kPlanWaves; ++w) count += hist[w * keys + tid];
    int total, n_used, n_items;
    const int first = block_scan(count, tmp, &total);
    const int at_used = block_scan(count > 0, tmp, &n_used);
    const int at_item = block_scan((count + kMultiItem - 1) / kMultiItem, tmp, &n_items);
    if (tid < n) {
        out.start[tid] = first;
        out.first_item[tid] = at_item;
        int p = first;
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = hist[w * keys + tid];
            hist[w * keys + tid] = p;
            p += c;
        }
        if (count > 0) {
            out.used[at_used] = tid;
            ends[at_used] = first + count;
            for (int k = 0; k * kMultiItem < count; ++k)
                out.items[at_item + k] = MultiItem{tid, first + k * kMultiItem, count - k * kMultiItem, k};
        }
    }
    for (int i = n_items + tid; i < max_items; i += kPlanThreads) out.items[i] = MultiItem{-1, 0, 0, 0};
    if (tid == 0) {
        out.start[n] = total;
        int p = total;
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = hist[w * keys + n];
            hist[w * keys + n] = p;
            p += c;
        }
        out.head[0] = n_used;
        out.head[1] = n_items;
        out.head[2] = total;
        out.head[3] = n;
    }
    __syncthreads();
    for (int t = t0; t < t1; t += 64) {
        const bool ok = t + lane < t1;
        const int id = ok ? ids[t + lane] : -1;
        const int key = id >= 0 && id < n ? id : n;
        const unsigned long long same = same_key(key, ok);
        int base = 0;
        if (ok) base = row[key];
        // every lane has read its base before the first lane of each id moves it on, and every
        // lane sees that before its next read
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (ok) {
            out.order[base + __popcll(same & below)] = t + lane;
            if ((same & below) == 0) row[key] = base + __popcll(same);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    // tile t covers positions [256 t, 256 t + 256): the adapters in use whose end lies past
    // its first position, up to the one that holds (or ends at) its last
    const int tiles = (M + kMultiTile - 1) / kMultiTile;
    for (int t = tid; t < tiles; t += kPlanThreads) {
        auto first_past = [&](int pos) {               // first k with ends[k] > pos
            int lo = 0, hi = n_used;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (ends[mid] > pos) hi = mid; else lo = mid + 1;
            }
            return lo;
        };
        const int p0 = t * kMultiTile, p1 = min(p0 + kMultiTile, total);
        const int k0 = first_past(p0);
        const int k1 = p1 > p0 ? min(n_used, first_past(p1 - 1) + 1) : k0;
        out.tile[t] = int2{k0, k1};
    }
}

struct Offsets { int64_t order, start, first_item, used, tile, items, words; };

Offsets offsets_of(int64_t M, int64_t n) {
    auto up = [](int64_t v) { return (v + 3) / 4 * 4; };
    Offsets o{};
    o.order = 4;
    o.start = o.order + up(M);
    o.first_item = o.start + up(n + 1);
    o.used = o.first_item + up(n);
    o.tile = o.used + up(n < M ? n : M);
    o.items = o.tile + up(2 * ((M + kMultiTile - 1) / kMultiTile));
    o.words = o.items + 4 * multi_max_items(M, n);
    return o;
}

}  // namespace

int64_t multi_plan_words(int64_t M, int64_t n) { return offsets_of(M, n).words; }

MultiPlan multi_plan_at(const void* buf, int64_t M, int64_t n) {
    const Offsets o = offsets_of(M, n);
    const int32_t* w = static_cast<const int32_t*>(buf);
    return MultiPlan{w, w + o.order, w + o.start, w + o.first_item, w + o.used, reinterpret_cast<const int2*>(w + o.tile),
                     reinterpret_cast<const MultiItem*>(w + o.items)};
}

hipError_t launch_multi_plan(const int32_t* ids, int64_t M, int n, void* buf, hipStream_t st) {
    const Offsets o = offsets_of(M, n);
    int32_t* w = static_cast<int32_t*>(buf);
    const PlanOut out{w, w + o.order, w + o.start, w + o.first_item, w + o.used,
                      reinterpret_cast<int2*>(w + o.tile), reinterpret_cast<MultiItem*>(w + o.items)};
    QN_LAUNCH("multi_plan_kernel", st, multi_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, ids,
              static_cast<int>(M), n, static_cast<int>(multi_max_items(M, n)), out);
    return hipGetLastError();
}

}  // namespace qn
