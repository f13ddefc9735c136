// embed.cu -- embedding lookup with scaling, and the gradient of its table.
//
//   out_i = E[id_i] scale,       dE[v] = scale sum_{i: id_i = v} dout_i
//
// The gradient sorts the tokens by id (stable, so that the order of a sum is that of
// the tokens), takes the sorted list in chunks of equal length, however often an id
// comes, sums each run of one id within a chunk in fp32, and joins the runs that go
// across chunks.  No floating-point sum depends on the order of arrivals; the same bits in
// every call.
//
// Bound by memory where tables and batches are large.  Measured on one GB300 (6772 GB/s copied):
// lookup 65536 x 4096 bf16 from 32000 rows 104 us, 6.2 TB/s (rows in blocks as they come; in
// blocks that stay 117 us).  Gradient of 65536 tokens added to 32000 x 4096 fp32 208 us, 4.7 TB/s:
// some 25 us of it sort.  8192 tokens, 50257 x 768 bf16 27 us for a floor of 13: filling 77 MB with
// zeros takes 12 to 15, the sums after it wait for their loads one after the other.  (Leaving
// part of the zeros to the sums' launch: 31 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "cluster_counts.h"
#include "run_reach.h"
#include "zs_internal.h"

namespace {

#include "step_common.cuh"
#include "step_end.cuh"
#include "loss_common.cuh"
#include "elem.cuh"
#include "launch.cuh"

[[maybe_unused]] constexpr uint32_t kSiteEmbed = 19, kSiteSort = 20, kSiteTable = 21;

constexpr int64_t kMaxTokens = 1 << 28, kMaxVocab = 1 << 30, kMaxWidth = 1 << 24;

struct EmbedArgs {
    const void* table;
    const int64_t* ids;
    int64_t tokens, vocab, width, table_stride;
    float scale;
    void* out;
    int64_t out_stride;
    const void* dout;
    int64_t dout_stride;
    void* dtable;
    int64_t dtable_stride;
    int32_t accumulate;
    // the tokens sorted by id, and the list's second place (sort passes write the two
    // in turn); ids outside the vocabulary count as `vocab` and come last
    uint32_t *keys, *places, *other_keys, *other_places;
    int32_t passes, bits;  // of the sort, and of a pass
    float* part;           // sums of runs that go across chunks: two rows to a chunk
    int32_t chunk;         // tokens of a chunk
    uint32_t* arrived;     // of the chunks that a run goes across, by the one it starts in and columns
    int64_t arrivals;      // how many of those counts
};

// ------------------------------------------------------------------- lookup ---

constexpr int kThreads = 256;

// (Rows written for another kernel to read once: they leave the table its place in L2.)
template <typename T, int V>
__device__ __forceinline__ void store_stream(Pack<T, V>* to, const Pack<T, V>& x) {
    if constexpr (sizeof(x) == 16)
        __stcs(&to->raw, x.raw);
    else
        *to = x;
}

// A team of `warps` warps copies a row, four vectors to a thread at a time.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) embed_kernel(const __grid_constant__ EmbedArgs a, int32_t warps) {
    const int threads = 32 * warps, teams = kThreads / threads, thread = threadIdx.x % threads;
    const int64_t vectors = a.width / V;
    griddep_wait();
    for (int64_t i = (int64_t)blockIdx.x * teams + threadIdx.x / threads; i < a.tokens; i += (int64_t)gridDim.x * teams) {
        const int64_t v = a.ids[i];
        const bool inside = v >= 0 && v < a.vocab;
        const Pack<T, V>* row = reinterpret_cast<const Pack<T, V>*>((const T*)a.table + (inside ? v : 0) * a.table_stride);
        Pack<T, V>* out = reinterpret_cast<Pack<T, V>*>((T*)a.out + i * a.out_stride);
        for (int64_t k0 = thread; k0 < vectors; k0 += 4 * threads) {
            Pack<T, V> x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (k0 + q * threads < vectors && inside) x[q] = row[k0 + q * threads];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t k = k0 + q * threads;
                if (k >= vectors || !ZS_RANGE_OK(kSiteEmbed, k * V, V, a.width)) break;
                float f[V];
                if (!inside) {
#pragma unroll
                    for (int j = 0; j < V; ++j) f[j] = 0.0f;
                    x[q] = pack<T, V>(f);
                } else if (a.scale != 1.0f) {
                    unpack<T, V>(x[q], f);
#pragma unroll
                    for (int j = 0; j < V; ++j) f[j] *= a.scale;
                    x[q] = pack<T, V>(f);
                }
                store_stream(out + k, x[q]);
            }
        }
    }
}

// --------------------------------------------------------------------- sort ---

constexpr int kAhead = 8;  // loads of 32 tokens that a warp has under way
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortCtas = 8, kMaxBits = 9, kBins = 1 << kMaxBits;
constexpr int kSortShared = (kSortWarps * kBins + 2 * kBins) * 4;

// The lanes of the warp with the same digit (those of `in`): a vote for each bit.  (The
// instruction that matches values took 70 cycles of the SM; nine votes take some 10.)
__device__ __forceinline__ uint32_t same_digit(uint32_t d, bool in) {
    uint32_t same = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < kMaxBits; ++b) {  // (bits that the digit does not have are 0 in all lanes)
        const bool set = (d & (1u << b)) != 0;
        const uint32_t votes = __ballot_sync(0xffffffffu, set);
        same &= set ? votes : ~votes;
    }
    return same;
}

// Cluster 0 sorts: passes of `bits` bits of the id from the lowest up.  A warp has a
// piece of the list, in order; in a pass it counts its digits, the counts turn into
// places (warps below, CTAs below, smaller digits), and it puts its tokens there, equal
// digits in their order.  The other clusters fill the table with zeros meanwhile.
// A cluster of eight has its counts one distributed-shared-memory read apart, and its
// barrier is the only one on the way.
template <typename G, int V>
__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const __grid_constant__ EmbedArgs a) {
    extern __shared__ uint32_t s_sort[];
    uint32_t(*const count)[kBins] = reinterpret_cast<uint32_t(*)[kBins]>(s_sort);  // of each warp
    uint32_t* const total = s_sort + kSortWarps * kBins;                            // of this CTA
    uint32_t* const base = total + kBins;
    __shared__ uint32_t s_scan[kSortWarps];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x >= kSortCtas) {
        if (a.accumulate) return;
        float zero[V] = {};
        const Pack<G, V> z = pack<G, V>(zero);
        // (rows that lie end to end are one)
        const bool flat = a.dtable_stride == a.width;
        if (flat) {
            const int64_t vectors = a.vocab * (a.width / V), step = (int64_t)(gridDim.x - kSortCtas) * kSortThreads;
            Pack<G, V>* const table = reinterpret_cast<Pack<G, V>*>(a.dtable);
            for (int64_t k = (int64_t)(blockIdx.x - kSortCtas) * kSortThreads + threadIdx.x; k < vectors; k += step)
                if (ZS_RANGE_OK(kSiteTable, k * V, V, a.vocab * a.width)) table[k] = z;
            return;
        }
        const int64_t vectors = a.width / V, step = (int64_t)(gridDim.x - kSortCtas) * kSortWarps;
        for (int64_t v = (int64_t)(blockIdx.x - kSortCtas) * kSortWarps + warp; v < a.vocab; v += step) {
            Pack<G, V>* row = reinterpret_cast<Pack<G, V>*>((G*)a.dtable + v * a.dtable_stride);
            for (int64_t k = lane; k < vectors; k += 32)
                if (ZS_RANGE_OK(kSiteTable, v, 1, a.vocab)) row[k] = z;
        }
        return;
    }
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < a.arrivals; i += kSortCtas * kSortThreads)
        a.arrived[i] = 0u;
    const uint32_t rank = cluster_rank();
    const int64_t me = (int64_t)rank * kSortWarps + warp, warps = kSortCtas * kSortWarps;
    const int64_t from = a.tokens * me / warps, to = a.tokens * (me + 1) / warps;
    const int bins = 1 << a.bits;
    for (int pass = 0; pass < a.passes; ++pass) {
        // the last pass writes keys, places
        const bool first = pass == 0, even = ((a.passes - 1 - pass) & 1) == 0;
        uint32_t *to_key = even ? a.keys : a.other_keys, *to_place = even ? a.places : a.other_places;
        const uint32_t *from_key = even ? a.other_keys : a.keys, *from_place = even ? a.other_places : a.places;
        const int shift = pass * a.bits;
        auto key_of = [&](int64_t i) {
            if (!first) return from_key[i];
            const int64_t v = a.ids[i];
            return v >= 0 && v < a.vocab ? (uint32_t)v : (uint32_t)a.vocab;
        };
        auto digit_of = [&](uint32_t key) { return (key >> shift) & (uint32_t)(bins - 1); };
        for (int b = lane; b < bins; b += 32) count[warp][b] = 0;
        __syncwarp();
        for (int64_t i0 = from; i0 < to; i0 += 32 * kAhead) {
            uint32_t key[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) key[q] = i0 + 32 * q + lane < to ? key_of(i0 + 32 * q + lane) : 0u;
#pragma unroll
            for (int q = 0; q < kAhead; ++q)
                if (i0 + 32 * q + lane < to) atomicAdd(&count[warp][digit_of(key[q])], 1u);
        }
        __syncthreads();
        uint32_t mine = 0;
        if (threadIdx.x < bins) {
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = count[w][threadIdx.x];
                count[w][threadIdx.x] = mine;
                mine += c;
            }
            total[threadIdx.x] = mine;
        }
        cluster_arrive();
        cluster_wait();
        uint32_t below = 0, all = 0;
        if (threadIdx.x < bins) {
            for (uint32_t c = 0; c < kSortCtas; ++c) {
                uint32_t at, x;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(total + threadIdx.x)), "r"(c));
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
                below += c < rank ? x : 0;
                all += x;
            }
        }
        // smaller digits
        uint32_t scan = all;
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += x;
        }
        if (lane == 31) s_scan[warp] = scan;
        __syncthreads();
        for (int w = 0; w < warp; ++w) scan += s_scan[w];
        if (threadIdx.x < bins) base[threadIdx.x] = scan - all + below;
        __syncthreads();
        for (int64_t i0 = from; i0 < to; i0 += 32 * kAhead) {
            uint32_t key[kAhead], place[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int64_t i = i0 + 32 * q + lane;
                key[q] = i < to ? key_of(i) : 0u;
                place[q] = first ? (uint32_t)i : i < to ? from_place[i] : 0u;
            }
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                if (i0 + 32 * q >= to) break;
                const bool in = i0 + 32 * q + lane < to;
                const uint32_t d = digit_of(key[q]), same = same_digit(d, in);
                if (in) {
                    const int64_t at = base[d] + count[warp][d] + (uint32_t)__popc(same & ((1u << lane) - 1u));
                    if (ZS_RANGE_OK(kSiteSort, at, 1, a.tokens)) {
                        to_key[at] = key[q];
                        to_place[at] = place[q];
                    }
                }
                __syncwarp();
                if (in && __ffs(same) - 1 == lane) count[warp][d] += __popc(same);
                __syncwarp();
            }
        }
        // (every CTA's writes, seen by every CTA; and the totals may be written again)
        cluster_arrive();
        cluster_wait();
    }
}

// ---------------------------------------------------------------------- sums ---

constexpr int kMaxChunk = 64;

template <int V>
__device__ __forceinline__ void add_in_memory(float* to, const float* x) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to + i), "f"(x[i]), "f"(x[i + 1]), "f"(x[i + 2]),
                         "f"(x[i + 3]) : "memory");
    } else if constexpr (V == 2) {
        asm volatile("red.global.add.v2.f32 [%0], {%1, %2};" ::"l"(to), "f"(x[0]), "f"(x[1]) : "memory");
    } else {
        asm volatile("red.global.add.f32 [%0], %1;" ::"l"(to), "f"(x[0]) : "memory");
    }
}
template <typename G, int V>
__device__ __forceinline__ void add_to_table(const EmbedArgs& a, uint32_t key, int64_t k, const float* sum) {
    if (!ZS_RANGE_OK(kSiteTable, key, 1, a.vocab)) return;
    Pack<G, V>* to = reinterpret_cast<Pack<G, V>*>((G*)a.dtable + (int64_t)key * a.dtable_stride + k);
    if constexpr (sizeof(G) == 4) {
        // added in L2: nothing waits for the row (an element is added to once in a call, so
        // no order can matter).  The same additions whatever the row's boundary allows to go out together.
        if (a.accumulate) {
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = __fmul_rn(sum[i], a.scale);
            add_in_memory<V>(reinterpret_cast<float*>(to), y);
            return;
        }
    }
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 0.0f;
    if (a.accumulate) unpack<G, V>(*to, x);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = fmaf(sum[i], a.scale, x[i]);
    *to = pack<G, V>(x);
}
// Where the sum of a run that goes across chunks waits: what continues a run from the
// chunk before in the chunk's first row, the start of one that goes on in its second.
template <int V>
__device__ __forceinline__ Pack<float, V>* part_at(const EmbedArgs& a, int64_t chunk, bool start, int64_t k) {
    return reinterpret_cast<Pack<float, V>*>(a.part + (2 * chunk + (start ? 1 : 0)) * a.width + k);
}

template <int V>
__device__ __forceinline__ Pack<float, V> load_part(const Pack<float, V>* p) {  // (written by other blocks: from L2)
    Pack<float, V> x;
    if constexpr (V == 8) {
        x.raw.a = __ldcg(&p->raw.a);
        x.raw.b = __ldcg(&p->raw.b);
    } else {
        x.raw = __ldcg(&p->raw);
    }
    return x;
}
// Adds up a run that goes across chunks once all of them have left their part: the block
// that comes last does, in the chunks' order.  Called by the whole block.
template <typename G, int V>
__device__ __noinline__ void join_run(const EmbedArgs& a, int64_t chunks, int32_t columns, int64_t c, uint32_t key, bool started_before,
                         int32_t column, int64_t q) {
    __shared__ int64_t s_first, s_last;
    __shared__ bool s_done;
    const int64_t vectors = a.width / V;
    __threadfence();  // (the block's part, before it is counted)
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        // chunks whose first token has the key, and the one that the run starts in
        auto goes_on = [&](int64_t j) { return j >= 0 && j < chunks && a.keys[j * a.chunk] == key; };
        int64_t first = c;
        if (started_before) {
            first -= zs::run_reach([&](int64_t at, int64_t stride) {
                return __ballot_sync(0xffffffffu, goes_on(c - at - stride * (lane + 1)));
            });
            if (first > 0 && a.keys[first * a.chunk - 1] == key) --first;
        }
        const int64_t last = c + zs::run_reach([&](int64_t at, int64_t stride) {
            return __ballot_sync(0xffffffffu, goes_on(c + at + stride * (lane + 1)));
        });
        if (lane == 0) {
            s_first = first;
            s_last = last;
            s_done = atomicAdd(a.arrived + first * columns + column, 1u) == (uint32_t)(last - first);
            __threadfence();
        }
    }
    __syncthreads();
    const int64_t first = s_first, last = s_last;
    const bool done = s_done;
    __syncthreads();  // (the places may be written again)
    if (!done || q >= vectors) return;
    const int64_t k = q * V;
    float sum[V];
    unpack<float, V>(load_part<V>(part_at<V>(a, first, true, k)), sum);
    constexpr int kAtOnce = V == 8 ? 4 : 8;  // (8 of 8 floats: registers; 31 us for 27 in the batch case)
    for (int64_t j = first + 1; j <= last; j += kAtOnce) {
        Pack<float, V> x[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (j + u <= last) x[u] = load_part<V>(part_at<V>(a, j + u, false, k));
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (j + u > last) break;
            float f[V];
            unpack<float, V>(x[u], f);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] += f[i];
        }
    }
    add_to_table<G, V>(a, key, k, sum);
}

// A block takes a chunk of the sorted list and up to blockDim.x vectors of the width, eight
// tokens' vectors under way at once.
template <typename T, typename G, int V>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const __grid_constant__ EmbedArgs a, int64_t chunks, int32_t columns) {
    __shared__ uint32_t s_key[kMaxChunk + 2], s_place[kMaxChunk];
    const int64_t vectors = a.width / V;
    constexpr uint32_t kNone = 0xffffffffu;
    griddep_wait();
    for (int64_t work = blockIdx.x; work < chunks * columns; work += gridDim.x) {
        const int64_t c = work / columns;
        const int32_t column = (int32_t)(work - c * columns);
        const int64_t q = (int64_t)column * blockDim.x + threadIdx.x, first = c * a.chunk;
        const int32_t n = a.tokens - first < a.chunk ? (int32_t)(a.tokens - first) : a.chunk;
        __syncthreads();
        for (int t = threadIdx.x; t < n + 2; t += blockDim.x) {
            const int64_t i = first + t - 1;
            s_key[t] = i >= 0 && i < a.tokens ? a.keys[i] : kNone;
            if (t < n) s_place[t] = a.places[first + t];
        }
        __syncthreads();
        if (q < vectors) {
            const int64_t k = q * V;
            const T* const rows = (const T*)a.dout + k;
            float sum[V];
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] = 0.0f;
            bool from_before = s_key[0] == s_key[1];
            for (int t0 = 0; t0 < n; t0 += 8) {
                Pack<T, V> x[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (t0 + u < n && s_key[t0 + u + 1] < (uint32_t)a.vocab)
                        x[u] = *reinterpret_cast<const Pack<T, V>*>(rows + (int64_t)s_place[t0 + u] * a.dout_stride);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int t = t0 + u;
                    if (t >= n) break;
                    const uint32_t key = s_key[t + 1];
                    if (key >= (uint32_t)a.vocab) break;
                    float f[V];
                    unpack<T, V>(x[u], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[i] += f[i];
                    const bool more = s_key[t + 2] == key;
                    if (more && t + 1 < n) continue;
                    // the run's end, here or at the chunk's
                    if (from_before || more)
                        *part_at<V>(a, c, !from_before, k) = pack<float, V>(sum);
                    else
                        add_to_table<G, V>(a, key, k, sum);
                    from_before = false;
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
                }
            }
        }
        // runs that go across chunks: the one from before, and one that starts here and goes on
        const uint32_t head = s_key[1], tail = s_key[n];
        const bool from_before = s_key[0] == head && head < (uint32_t)a.vocab;
        const bool goes_on = s_key[n + 1] == tail && tail < (uint32_t)a.vocab && !(from_before && head == tail);
        if (from_before) join_run<G, V>(a, chunks, columns, c, head, true, column, q);
        if (goes_on) join_run<G, V>(a, chunks, columns, c, tail, false, column, q);
    }
}

// ------------------------------------------------------------------- launches ---

// Tokens of a chunk, a power of 2: few where there are few tokens, for more blocks (some 1200,
// each of up to 1024 of the width); many where there are enough blocks, for fewer parts of runs.
int32_t chunk_of(int64_t tokens, int64_t width) {
    const int64_t blocks = tokens * (width > 1024 ? width / 1024 : 1);
    int32_t chunk = tokens >= 8192 ? 16 : 8;
    while (chunk < kMaxChunk && (int64_t)chunk * 1216 < blocks) chunk *= 2;
    return chunk;
}

// With two tokens and more to an id some runs are long, and the longest chain of loads is a
// chunk's tokens, eight at a time, then the parts of the most frequent id, four (of eight floats)
// or eight at a time.  Where that id has a tenth of the tokens the chain is least for chunks of
// some sqrt(tokens / 5) or sqrt(tokens / 10); the rule takes sqrt(tokens / 8), from the sizes alone, whatever
// the ids.  (17133 tokens of 127 ids, 568 wide fp32: 26 us for 40; 9292 of 11420, 472 wide
// bf16: 32 for 26, so not there.  An id with more of the tokens waits for more parts: 65536
// tokens of one id, 1024 wide bf16, 180 us.)
int32_t chunk_of_runs(int64_t tokens, int64_t width, int64_t vocab) {
    int32_t chunk = chunk_of(tokens, width);
    if (tokens / 2 < vocab) return chunk;
    while (chunk < kMaxChunk && (int64_t)chunk * chunk * 8 < tokens) chunk *= 2;
    return chunk;
}

// The parts of the scratch buffer, as offsets (with the fewest tokens to a chunk).
struct Plan {
    int64_t list[4], part, arrived, arrivals, chunks, total;
};
Plan plan_of(int64_t tokens, int64_t width) {
    Plan p;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 127) / 128 * 128;
        return here;
    };
    for (int64_t& l : p.list) l = take(4 * tokens);
    const int32_t chunk = chunk_of(tokens, width);
    p.chunks = (tokens + chunk - 1) / chunk;
    p.part = take(8 * p.chunks * width);
    p.arrivals = p.chunks * ((width + kThreads - 1) / kThreads);
    p.arrived = take(4 * p.arrivals);
    p.total = at > 0 ? at : 128;
    return p;
}

// Whether every row starts on a boundary of `bytes` and has whole vectors of them.
bool vectors_fit(const void* p, int64_t stride, int64_t width, int64_t size, int64_t bytes = 16) {
    return zs::aligned_to(p, (uintptr_t)bytes) && stride * size % bytes == 0 && width * size % bytes == 0;
}

template <typename T, int V>
int32_t launch_lookup(const EmbedArgs& a, cudaStream_t stream) {
    const int64_t vectors = a.width / V;
    int warps = 1;
    while (warps < kThreads / 32 && vectors > 128ll * warps) warps *= 2;
    const int teams = kThreads / (32 * warps);
    const int64_t blocks = (a.tokens + teams - 1) / teams, most = 1 << 24;
    return launch(embed_kernel<T, V>, dim3((unsigned)(blocks < most ? blocks : most)), kThreads, stream, "embed_kernel", a, warps);
}

template <typename T, typename G, int V>
int32_t launch_grad(const EmbedArgs& a, int64_t chunks, cudaStream_t stream) {
    // the sort's cluster, and clusters that fill the other SMs with zeroing blocks
    const int most = clusters_of((const void*)embed_sort_kernel<G, V>, kSortThreads, kSortCtas, kSortShared);
    if (most < 1) return ZS_ERR_CUDA;
    ZS_TRY(launch_clusters(embed_sort_kernel<G, V>, a.accumulate ? 1 : most > 1 ? most : 2, kSortCtas, kSortThreads, kSortShared,
                           stream, a, "embed_sort_kernel"));
    if (chunks == 0) return ZS_OK;
    const int64_t vectors = a.width / V;
    const int threads = vectors < kThreads ? (int)((vectors + 31) / 32 * 32) : kThreads;
    const int32_t columns = (int32_t)((vectors + threads - 1) / threads);
    // (a block to a chunk, as they come: chunks differ in their stores)
    const int64_t blocks = chunks * columns, limit = 1 << 24;
    return launch(embed_sum_kernel<T, G, V>, dim3((unsigned)(blocks < limit ? blocks : limit)), threads, stream, "embed_sum_kernel",
                  a, chunks, columns);
}

bool valid_stride(int64_t rows, int64_t width, int64_t stride) {
    return rows <= 1 || (stride >= width && stride <= 1ll << 40);
}

int32_t check_embed(const zs_embed* e) {
    if (e == nullptr || e->tokens < 0 || e->tokens > kMaxTokens || e->vocab < 1 || e->vocab > kMaxVocab || e->width < 1 ||
        e->width > kMaxWidth || (e->type != ZS_F32 && e->type != ZS_F16 && e->type != ZS_BF16) || e->reserved != 0 ||
        !(e->scale >= -1e30 && e->scale <= 1e30) || (e->tokens > 0 && e->ids == nullptr))
        return ZS_ERR_ARG;
    return zs::aligned_to(e->ids, 8) ? ZS_OK : ZS_ERR_ALIGN;
}
EmbedArgs args_of(const zs_embed* e) {
    EmbedArgs a = {};
    a.table = e->table;
    a.ids = e->ids;
    a.tokens = e->tokens;
    a.vocab = e->vocab;
    a.width = e->width;
    a.table_stride = e->vocab > 1 ? e->table_stride : e->width;
    a.scale = (float)e->scale;
    return a;
}

}  // namespace

namespace zs {
uint64_t take_fault_embed() { return take_fault(); }
}  // namespace zs

extern "C" {

ZS_API int32_t zero_embed_async(const zs_embed* e, void* out, int64_t out_stride, void* stream) {
    zs::NvtxRange nvtx_range("zero_embed_async");
    ZS_TRY(check_embed(e));
    if (e->tokens == 0) return ZS_OK;
    if (e->table == nullptr || out == nullptr || !valid_stride(e->vocab, e->width, e->table_stride) ||
        !valid_stride(e->tokens, e->width, out_stride))
        return ZS_ERR_ARG;
    const uintptr_t size = (uintptr_t)elem_size(e->type);
    if (!zs::aligned_to(e->table, size) || !zs::aligned_to(out, size)) return ZS_ERR_ALIGN;
    EmbedArgs a = args_of(e);
    a.out = out;
    a.out_stride = e->tokens > 1 ? out_stride : e->width;
    return with_elem(e->type, [&](auto t) {
        using T = decltype(t);
        auto fit = [&](int64_t bytes) {
            return vectors_fit(a.table, a.table_stride, a.width, sizeof(T), bytes) && vectors_fit(out, a.out_stride, a.width, sizeof(T), bytes);
        };
        if (fit(16)) return launch_lookup<T, 16 / sizeof(T)>(a, (cudaStream_t)stream);
        // (two elements of 16 bits to an access where rows allow it)
        return fit(4) ? launch_lookup<T, 4 / sizeof(T)>(a, (cudaStream_t)stream) : launch_lookup<T, 1>(a, (cudaStream_t)stream);
    });
}

ZS_API int64_t zero_embed_work_bytes(int64_t tokens, int64_t width) {
    if (tokens < 0 || tokens > kMaxTokens || width < 1 || width > kMaxWidth) return ZS_ERR_ARG;
    return plan_of(tokens, width).total;
}

ZS_API int32_t zero_embed_grad_async(const zs_embed* e, const void* dout, int64_t dout_stride, void* dtable,
                                     int64_t dtable_stride, int32_t dtable_type, int32_t accumulate, void* work_dev,
                                     int64_t work_bytes, void* stream) {
    zs::NvtxRange nvtx_range("zero_embed_grad_async");
    ZS_TRY(check_embed(e));
    if (dtable == nullptr || work_dev == nullptr || (dtable_type != e->type && dtable_type != ZS_F32) ||
        (accumulate != 0 && accumulate != 1) || (e->tokens > 0 && dout == nullptr) ||
        !valid_stride(e->tokens, e->width, dout_stride) || !valid_stride(e->vocab, e->width, dtable_stride) ||
        work_bytes < zero_embed_work_bytes(e->tokens, e->width))
        return ZS_ERR_ARG;
    if (!zs::aligned_to(dout, (uintptr_t)elem_size(e->type)) || !zs::aligned_to(dtable, (uintptr_t)elem_size(dtable_type)) ||
        !zs::aligned_to(work_dev, 16))
        return ZS_ERR_ALIGN;
    EmbedArgs a = args_of(e);
    a.dout = dout;
    a.dout_stride = e->tokens > 1 ? dout_stride : e->width;
    a.dtable = dtable;
    a.dtable_stride = e->vocab > 1 ? dtable_stride : e->width;
    a.accumulate = accumulate;
    if (accumulate && e->tokens == 0) return ZS_OK;
    const Plan p = plan_of(e->tokens, e->width);
    uint32_t** const lists[] = {&a.keys, &a.places, &a.other_keys, &a.other_places};
    for (int i = 0; i < 4; ++i) *lists[i] = (uint32_t*)((char*)work_dev + p.list[i]);
    a.part = (float*)((char*)work_dev + p.part);
    a.chunk = chunk_of_runs(e->tokens, e->width, e->vocab);
    const int64_t chunks = (e->tokens + a.chunk - 1) / a.chunk;
    a.arrived = (uint32_t*)((char*)work_dev + p.arrived);
    a.arrivals = p.arrivals;
    int32_t bits = 1;  // of the largest key, `vocab`
    while (e->vocab >> bits != 0) ++bits;
    a.passes = (bits + kMaxBits - 1) / kMaxBits;
    a.bits = (bits + a.passes - 1) / a.passes;
    return with_elem(e->type, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto g) {
            using G = decltype(g);
            constexpr int V = 16 / sizeof(T);
            const bool wide = vectors_fit(dout, a.dout_stride, a.width, sizeof(T)) &&
                              vectors_fit(dtable, a.dtable_stride, a.width, sizeof(G));
            if (wide) return launch_grad<T, G, V>(a, chunks, (cudaStream_t)stream);
            if constexpr (sizeof(T) == 2)  // (two elements to an access where rows allow it)
                if (vectors_fit(dout, a.dout_stride, a.width, 2, 4) && vectors_fit(dtable, a.dtable_stride, a.width, sizeof(G), 2 * sizeof(G)))
                    return launch_grad<T, G, 2>(a, chunks, (cudaStream_t)stream);
            return launch_grad<T, G, 1>(a, chunks, (cudaStream_t)stream);
        };
        return dtable_type == ZS_F32 ? go(float()) : go(t);
    });
}

}  // extern "C"
